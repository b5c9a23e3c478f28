"""A second pass: a small language model that reads each lane's first-pass words
and goes on from them.

The model is a decoder-only transformer with grouped heads, whose matrices are
kept in 4-bit codes.  One step takes one token per lane through it: products
with the packed matrices, the heads' norm and rotation with the write into the
paged cache, attention over the cache, and the draw of the next token, all in
the CUDA library; what is left to torch are the embedding row, the norm between
layers and the gate.  A step is captured once as a CUDA graph that finds its
token, place and random number by a counter on the device, so a whole pass is
one graph launch per token and nothing is read back before its end.

Lanes need not be of one length: a lane reads its words one per step, then its
own tokens, and after its last one runs along with an empty cache view.

    lm = LanguageModel.random(Shape(vocab=5000))
    passes = SecondPass(lm, max_lanes=64, max_tokens=256)
    answers = passes.run([r["words"] for r in decoder.decode(lp, lens)], new_tokens=32, top_p=0.9)

Where hypotheses are rescored, all lanes may follow one prefix (an instruction,
the transcript so far), which is read once and kept in the cache once
(``read_prefix``); lanes may have low-rank adapters of their own, by speaker or
domain (``LanguageModel.adapt``); and ``score`` reads all words at once and
answers how likely each of them was.

    lm.adapt(tensors)
    passes.read_prefix(tokens)
    scores = passes.score(hypotheses, top=5, adapters=[speaker_of[h] for h in hypotheses])

``python -m wfst_beam_search_gb300.second_pass`` (in the source tree) decodes a
synthetic workload and runs such a pass, with random weights, on its words.
"""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np
import torch
import torch.nn.functional as F

from . import WFST_SCORE_TOP, _ops


@dataclass(frozen=True)
class Shape:
    """Sizes of a model.  ``start`` is the token before the first word;
    ``window`` and ``sinks`` limit what a token sees (0: everything)."""
    vocab: int
    width: int = 512
    layers: int = 4
    q_heads: int = 8
    kv_heads: int = 2
    head_dim: int = 64
    hidden: int = 1024
    group: int = 64
    window: int = 0
    sinks: int = 0
    start: int = 0
    eps: float = 1e-6
    base: float = 10000.0


def quantize(weight, group, dtype):
    """Codes uint8 [n, k / 2] and scales ``dtype`` [n, k / group] nearest to a
    matrix [n, k], for ``pack_quant`` without zero points."""
    n, k = weight.shape
    w = weight.float().reshape(n, k // group, group)
    scales = (w.abs().amax(2) / 7).clamp_min(2.0 ** -24).to(dtype)
    c = (w / scales.float()[:, :, None] + 8).round().clamp(0, 15).to(torch.uint8).reshape(n, k)
    return c[:, ::2] | c[:, 1::2] << 4, scales


class LanguageModel:
    """The weights: ``embed`` [vocab, width], ``layers`` of packed matrices and
    gains, the last ``gain`` and the packed ``head``."""

    def __init__(self, shape, tensors, dtype=torch.bfloat16, device="cuda"):
        """``tensors``: "embed" [vocab, width], "gain" [width], "head" [vocab,
        width], and for each layer i "i.gain1", "i.qkv" [(q_heads + 2 kv_heads)
        * head_dim, width], "i.q_gain", "i.k_gain" [head_dim], "i.out" [width,
        q_heads * head_dim], "i.gain2", "i.up" [2 hidden, width] (gate first),
        "i.down" [width, hidden], in any floating type."""
        s, heads = shape, shape.q_heads * shape.head_dim
        if not 0 <= s.start < s.vocab:
            raise ValueError(f"the start token {s.start} is outside the vocabulary of {s.vocab}")
        sizes = {"embed": (s.vocab, s.width), "gain": (s.width,), "head": (s.vocab, s.width)}
        for i in range(s.layers):
            sizes.update({f"{i}.gain1": (s.width,), f"{i}.gain2": (s.width,), f"{i}.q_gain": (s.head_dim,),
                          f"{i}.k_gain": (s.head_dim,), f"{i}.out": (s.width, heads),
                          f"{i}.qkv": (heads + 2 * s.kv_heads * s.head_dim, s.width),
                          f"{i}.up": (2 * s.hidden, s.width), f"{i}.down": (s.width, s.hidden)})
        for name, size in sizes.items():
            if name not in tensors or tuple(tensors[name].shape) != size:
                raise ValueError(f"{name} must be a tensor of shape {size}")

        def take(name):
            t = tensors[name].detach().to(device)
            if t.dim() == 1 or name == "embed":
                return t.to(dtype).contiguous()
            return _ops.pack_quant(*quantize(t, s.group, dtype))

        self.shape, self.dtype = shape, dtype
        self.embed, self.gain, self.head = take("embed"), take("gain"), take("head")
        self.adapters, self.adapter_count, self.adapter_scales = {}, 0, None
        self.device = self.embed.device    # with its number, whatever is the current device later
        self.layers = [{name: take(f"{i}.{name}") for name in
                        ("gain1", "qkv", "q_gain", "k_gain", "out", "gain2", "up", "down")} for i in range(s.layers)]

    @classmethod
    def random(cls, shape, seed=0, dtype=torch.bfloat16, device="cuda"):
        return cls(shape, random_tensors(shape, seed), dtype, device)

    def adapt(self, tensors, scales=None):
        """Low-rank adapters beside some matrices, in place of those before:
        "i.qkv.shrink" [count, rank, width] and "i.qkv.expand" [count, outputs,
        rank] add scales[a] * expand[a] @ shrink[a] to that matrix for the lanes
        of adapter a, and so do "out", "up" and "down".  One count for all;
        ``scales`` float [count], one by default."""
        s, heads = self.shape, self.shape.q_heads * self.shape.head_dim
        sizes = {"qkv": (heads + 2 * s.kv_heads * s.head_dim, s.width), "out": (s.width, heads),
                 "up": (2 * s.hidden, s.width), "down": (s.width, s.hidden)}
        known = {f"{i}.{m}.{part}" for i in range(s.layers) for m in sizes for part in ("shrink", "expand")}
        if not tensors or set(tensors) - known:
            raise ValueError(f"adapters of no matrix: {sorted(set(tensors) - known)}")
        count, adapters = len(next(iter(tensors.values()))), {}
        for i in range(s.layers):
            for m, (n, k) in sizes.items():
                pair = [tensors.get(f"{i}.{m}.{part}") for part in ("shrink", "expand")]
                if pair == [None, None]:
                    continue
                if any(p is None or p.dim() != 3 or len(p) != count for p in pair):
                    raise ValueError(f"{i}.{m} needs both parts of {count} adapters, [count, rank, {k}] and [count, {n}, rank]")
                rank = pair[0].shape[1]
                if pair[0].shape[2] != k or pair[1].shape[1:] != (n, rank) or rank % 8 or not 8 <= rank <= 128:
                    raise ValueError(f"{i}.{m}: [count, rank, {k}] and [count, {n}, rank], rank a multiple of 8 up to 128")
                adapters[i, m] = tuple(p.detach().to(self.device, self.dtype).contiguous() for p in pair)
        if scales is not None:
            scales = torch.as_tensor(scales).detach().to(self.device, torch.float32).contiguous()
            if tuple(scales.shape) != (count,):
                raise ValueError(f"scales must be [{count}]")
        self.adapters, self.adapter_count, self.adapter_scales = adapters, count, scales

    def product(self, x, layer, name, which):
        """x times a layer's matrix, with the adapters of ``which``."""
        y = _ops.matvec_quant(x, self.layers[layer][name])
        pair = self.adapters.get((layer, name))
        return y if pair is None else _ops.add_lowrank(y, x, *pair, which, self.adapter_scales, out=y)


def random_tensors(shape, seed=0):
    """Random weights of a model, as ``LanguageModel`` takes them."""
    s, g = shape, torch.Generator()
    g.manual_seed(seed)

    def matrix(n, k):
        return torch.randn(n, k, generator=g) * k ** -0.5

    heads = s.q_heads * s.head_dim
    t = {"embed": torch.randn(s.vocab, s.width, generator=g), "gain": torch.ones(s.width), "head": matrix(s.vocab, s.width)}
    for i in range(s.layers):
        t.update({f"{i}.gain1": torch.ones(s.width), f"{i}.gain2": torch.ones(s.width),
                  f"{i}.q_gain": torch.ones(s.head_dim), f"{i}.k_gain": torch.ones(s.head_dim),
                  f"{i}.qkv": matrix(heads + 2 * s.kv_heads * s.head_dim, s.width), f"{i}.out": matrix(s.width, heads),
                  f"{i}.up": matrix(2 * s.hidden, s.width), f"{i}.down": matrix(s.width, s.hidden)})
    return t


class SecondPass:
    """A model with its cache: up to ``max_lanes`` lanes of up to
    ``max_tokens`` tokens each (start, words and answer), whose pages come from
    one pool of ``pages`` (by default enough for all lanes at full length).
    ``rows``: how many words ``read_prefix`` and ``score`` take through the
    model at a time."""

    prefix, prefix_table, prefix_length, rows = 0, None, None, 256    # tokens of the prefix, its pages, its length on the device
    adapted = None    # the adapters in the graph

    def __init__(self, model, max_lanes, max_tokens, page_size=64, pages=None, rows=256):
        s, dev = model.shape, model.device
        self.model, self.lanes, self.max_tokens, self.page = model, max_lanes, max_tokens, page_size
        per_lane = -(-max_tokens // page_size)
        self.pages = max_lanes * per_lane if pages is None else pages
        self.cache = [torch.zeros(2, self.pages, page_size, s.kv_heads, s.head_dim, dtype=model.dtype, device=dev)
                      for _ in range(s.layers)]
        self.table = torch.zeros(max_lanes, per_lane, dtype=torch.int32, device=dev)
        self.rows = rows
        self.rotary = self._rotary(max_tokens)
        self.which = torch.full((max_lanes,), -1, dtype=torch.int32, device=dev)    # each lane's adapter
        # what the steps of a pass take: token (-1: the one drawn before), position, slot, length
        self.plan = torch.zeros(max_tokens, 4, max_lanes, dtype=torch.int32, device=dev)
        self.uniform = torch.zeros(max_tokens, max_lanes, device=dev)
        self.settings = {name: torch.zeros(max_lanes, device=dev, dtype=torch.int32 if name == "top_k" else torch.float32)
                         for name in ("temperature", "top_k", "top_p", "min_p")}
        self.drawn = torch.zeros(max_tokens, max_lanes, dtype=torch.int32, device=dev)
        self.logprobs = torch.zeros(max_tokens, max_lanes, device=dev)
        self.last = torch.zeros(max_lanes, dtype=torch.int32, device=dev)
        self.at = torch.zeros(1, dtype=torch.int64, device=dev)
        self.workspace = _ops.attend_workspace(dev)
        self.graph = None

    def _rotary(self, contexts):
        s = self.model.shape
        angle = (torch.arange(contexts, dtype=torch.float64)[:, None]
                 * s.base ** (-torch.arange(0, s.head_dim, 2, dtype=torch.float64) / s.head_dim))
        return torch.cat([angle.cos(), angle.sin()], 1).float().to(self.model.device)

    def logits(self, tokens, positions, slots, lengths):
        """One token per lane through the model; its keys and values are put
        into the cache.  int32 [lanes] each; a lane with slot -1 and length 0
        is idle.  (Positions count the prefix, if there is one; lengths do not.)"""
        x = self._through(tokens, positions, slots, lengths, self.table, self.which, self.prefix_length)
        return _ops.matvec_quant(x, self.model.head)

    def _through(self, tokens, positions, slots, lengths, table, which, prefix_length):
        """Tokens through the model up to the head, each in its own row: those of
        one lane may be rows of one call, since a layer's keys and values are in
        the cache before any of its rows attends."""
        m, s, rows = self.model, self.model.shape, tokens.shape[0]
        hq, hkv = s.q_heads, s.kv_heads
        x = F.embedding(tokens, m.embed)
        for i, (layer, (keys, values)) in enumerate(zip(m.layers, self.cache)):
            h = m.product(F.rms_norm(x, (s.width,), layer["gain1"], s.eps), i, "qkv", which)
            h = h.view(rows, hq + 2 * hkv, s.head_dim)
            q = _ops.norm_rotate(h[:, :hq], h[:, hq:hq + hkv], h[:, hq + hkv:], positions, self.rotary,
                                 layer["q_gain"], layer["k_gain"], keys, values, slots, eps=s.eps)
            if prefix_length is None:
                o = _ops.attend_paged(q, keys, values, table, lengths, window=s.window, sinks=s.sinks,
                                      workspace=self.workspace)
            else:
                o = _ops.attend_prefix(q, keys, values, self.prefix_table, prefix_length, table, lengths,
                                       workspace=self.prefix_workspace)
            x = x + m.product(o.view(rows, -1), i, "out", which)
            h = m.product(F.rms_norm(x, (s.width,), layer["gain2"], s.eps), i, "up", which)
            x = x + m.product(F.silu(h[:, :s.hidden]) * h[:, s.hidden:], i, "down", which)
        return F.rms_norm(x, (s.width,), m.gain, s.eps)

    def read_prefix(self, tokens):
        """Reads ``tokens`` into the cache, for all lanes of the passes that
        follow to go on from; they take pages from the pool's end.  None: no
        prefix any more.  (A prefix is read with no adapter.)"""
        s, dev, page = self.model.shape, self.model.device, self.page
        tokens = [] if tokens is None else [int(t) for t in tokens]
        if tokens and s.window:
            raise ValueError("a model with a window reads no prefix")
        if any(not 0 <= t < s.vocab for t in tokens):
            raise ValueError("the prefix has a token outside the vocabulary")
        need = -(-len(tokens) // page)
        if need > self.pages:
            raise ValueError(f"the prefix takes {need} pages, the pool has {self.pages}")
        self.graph, self.prefix = None, len(tokens)    # (the step is another one)
        self.rotary = self._rotary(self.prefix + self.max_tokens)
        if not tokens:
            self.prefix_table = self.prefix_length = self.prefix_workspace = None
            return
        with torch.cuda.device(dev):
            self.prefix_table = torch.arange(self.pages - need, self.pages, dtype=torch.int32, device=dev)
            self.prefix_length = torch.zeros(1, dtype=torch.int32, device=dev)
            self.prefix_workspace = _ops.attend_prefix_workspace(max(self.lanes, self.rows, page), s.q_heads, s.kv_heads,
                                                                 s.head_dim, dev)
            # so many whole pages at a time, behind those that have been read
            step = max(1, self.rows // page) * page
            for first in range(0, len(tokens), step):
                n = min(step, len(tokens) - first)
                at = torch.arange(first, first + n, dtype=torch.int32, device=dev)
                pages = self.prefix_table[first // page:-(-(first + n) // page)]
                self.prefix_length.fill_(first)
                self._through(torch.tensor(tokens[first:first + n], dtype=torch.int32, device=dev), at,
                              self.prefix_table[0] * page + at, at - first + 1, pages.expand(n, -1),
                              torch.full_like(at, -1), self.prefix_length)
            self.prefix_length.fill_(len(tokens))

    def _step(self):
        tokens, positions, slots, lengths = self.plan.index_select(0, self.at)[0]
        # (a lane whose logits were all NaN drew -1: it goes on from token 0, and ``run`` ends its answer)
        tokens = torch.where(tokens < 0, self.last.clamp_min(0), tokens)
        drawn, logprobs, _ = _ops.sample_tokens(self.logits(tokens, positions, slots, lengths),
                                                self.uniform.index_select(0, self.at)[0], **self.settings)
        self.last.copy_(drawn)
        self.drawn.index_copy_(0, self.at, drawn[None])
        self.logprobs.index_copy_(0, self.at, logprobs[None])
        self.at.add_(1)

    def _capture(self):
        """The step as a graph, after one that only idle lanes take part in.
        The model's device is the current one."""
        self._load(np.zeros((1, 4, self.lanes), np.int32) + np.array([0, 0, -1, 0], np.int32)[None, :, None])
        side = torch.cuda.Stream(self.model.device)
        side.wait_stream(torch.cuda.current_stream(self.model.device))
        with torch.cuda.stream(side):
            self._step()
        torch.cuda.current_stream(self.model.device).wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):    # (torch's own capture stream may be another device's)
            self._step()
        self.graph, self.adapted = graph, getattr(self.model, "adapters", None)

    def _load(self, plan):
        self.plan[:len(plan)].copy_(torch.from_numpy(np.ascontiguousarray(plan)))
        self.at.zero_()

    def plan_lanes(self, words, new_tokens):
        """(plan [steps, 4, lanes], page table) of a pass, pages in the order
        of need."""
        if len(words) > self.lanes:
            raise ValueError(f"{len(words)} lanes, made for {self.lanes}")
        if new_tokens < 1:
            raise ValueError("new_tokens must be >= 1")
        lens = [len(w) + new_tokens for w in words]    # the start token in, the last token out
        if max(lens, default=0) > self.max_tokens:
            raise ValueError(f"a lane takes {max(lens)} tokens, made for {self.max_tokens}")
        need = [-(-n // self.page) for n in lens]
        left = self.pages - -(-self.prefix // self.page)
        if sum(need) > left:
            raise ValueError(f"the lanes take {sum(need)} pages, the pool has {left}")
        plan = np.zeros((max(lens, default=0), 4, self.lanes), np.int32)
        plan[:, 2] = -1
        table = np.zeros(self.table.shape, np.int32)
        page = 0
        for p in range(table.shape[1]):
            for b, n in enumerate(need):
                if p < n:
                    table[b, p] = page
                    page += 1
        for b, n in enumerate(lens):
            if any(not 0 <= w < self.model.shape.vocab for w in words[b]):
                raise ValueError(f"lane {b} has a word outside the vocabulary")
            at = np.arange(n)
            plan[:n, 0, b] = -1
            plan[:len(words[b]) + 1, 0, b] = [self.model.shape.start, *words[b]]
            plan[:n, 1, b] = self.prefix + at
            plan[:n, 2, b] = table[b, at // self.page] * self.page + at % self.page
            plan[:n, 3, b] = at + 1
        return plan, table

    def _adapters(self, words, adapters):
        """Each lane's adapter, -1 for none."""
        count = getattr(self.model, "adapter_count", 0)
        which = [-1] * len(words) if adapters is None else [-1 if a is None else int(a) for a in adapters]
        if len(which) != len(words) or any(not -1 <= a < count for a in which):
            raise ValueError(f"adapters must be one number below {count}, or None, for each lane")
        return which

    def score(self, words, top=0, adapters=None):
        """How likely each lane's ``words`` are: [{"logprobs", "entropy"}, ...],
        a number for each word, and with ``top`` also "alternatives", the `top`
        likeliest (token, logprob) in its place.  ``adapters`` as for ``run``."""
        if not 0 <= top <= WFST_SCORE_TOP:
            raise ValueError(f"top must be between 0 and {WFST_SCORE_TOP}")
        answers = [{"logprobs": [], "entropy": [], **({"alternatives": []} if top else {})} for _ in words]
        for lanes, targets, logits in self._read(words, adapters):
            got = [t.cpu() for t in _ops.score_tokens(logits, targets, top=top)]
            for b, lp, e, tokens, logprobs in zip(lanes, *(t.tolist() for t in got)):
                answers[b]["logprobs"].append(lp)
                answers[b]["entropy"].append(e)
                if top:
                    answers[b]["alternatives"].append(list(zip(tokens, logprobs)))
        return answers

    def _read(self, words, adapters=None):
        """(lane of each row, the word to come int32 [rows], logits [rows, vocab])
        for every word of all lanes, ``self.rows`` of them at a time."""
        which = self._adapters(words, adapters)
        if not any(len(w) for w in words):
            return
        plan, table = self.plan_lanes(words, 1)
        dev = self.model.device
        rows = [(b, i) for b, w in enumerate(words) for i in range(len(w))]
        with torch.cuda.device(dev):
            table = torch.from_numpy(table).to(dev)
            for first in range(0, len(rows), self.rows):
                some = rows[first:first + self.rows]
                b, i = (np.array(v) for v in zip(*some))
                tokens, positions, slots, lengths = torch.from_numpy(np.ascontiguousarray(plan[i, :, b].T)).to(dev)
                lanes = torch.from_numpy(b).to(dev)
                x = self._through(tokens, positions, slots, lengths, table[lanes],
                                  torch.tensor(which, dtype=torch.int32, device=dev)[lanes], self.prefix_length)
                targets = torch.tensor([words[c][j] for c, j in some], dtype=torch.int32, device=dev)
                yield b.tolist(), targets, _ops.matvec_quant(x, self.model.head)

    def run(self, words, new_tokens, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, seed=0, graph=True, adapters=None):
        """Read each lane's ``words`` and draw ``new_tokens`` tokens after
        them: [{"tokens", "logprobs"}, ...].  The same seed draws the same.
        ``adapters``: each lane's adapter (see ``LanguageModel.adapt``) or None.
        An answer ends where its logits hold no number (weights or activations
        that left the type's range): tokens -1, logprobs -inf from there on."""
        # (``sample_tokens`` refuses numbers, but here they reach it as a value per lane)
        for name, fits in (("temperature", 0 <= temperature <= 3e38), ("top_k", 0 <= top_k < 2 ** 31), ("top_p", top_p > 0),
                           ("min_p", 0 <= min_p <= 1)):
            if not fits:
                raise ValueError(f"{name} is out of range")
        which = self._adapters(words, adapters)
        plan, table = self.plan_lanes(words, new_tokens)
        if not len(plan):
            return []
        with torch.cuda.device(self.model.device):    # streams, capture and replay are of the current device
            # (a graph holds the addresses of the adapters that it was made with)
            if graph and (self.graph is None or self.adapted is not getattr(self.model, "adapters", None)):
                self._capture()
            self._load(plan)
            self.table.copy_(torch.from_numpy(table))
            if getattr(self.model, "adapter_count", 0):
                self.which.copy_(torch.tensor(which + [-1] * (self.lanes - len(which)), dtype=torch.int32))
            g = torch.Generator()
            g.manual_seed(seed)
            self.uniform[:len(plan)].copy_(torch.rand(len(plan), self.lanes, generator=g))
            for name, value in (("temperature", temperature), ("top_k", top_k), ("top_p", top_p), ("min_p", min_p)):
                self.settings[name].fill_(value)
            for _ in range(len(plan)):
                self.graph.replay() if graph else self._step()
        drawn, logprobs = self.drawn[:len(plan)].cpu().numpy(), self.logprobs[:len(plan)].cpu().numpy()
        answers = []
        for b, w in enumerate(words):
            t, lp = drawn[len(w):len(w) + new_tokens, b], logprobs[len(w):len(w) + new_tokens, b]
            ended = np.logical_or.accumulate(t < 0)
            answers.append({"tokens": np.where(ended, -1, t).tolist(), "logprobs": np.where(ended, -np.inf, lp).tolist()})
        return answers


def main():
    import argparse
    import time

    import synth

    import wfst_beam_search_gb300 as W

    ap = argparse.ArgumentParser(description="first pass on a synthetic workload, second pass on its words")
    ap.add_argument("--workload", type=int, default=1, help="index of the synthetic workload")
    ap.add_argument("--new-tokens", type=int, default=32)
    ap.add_argument("--top-p", type=float, default=0.9)
    ap.add_argument("--prefix", type=int, default=0, help="tokens of a (random) prefix that all lanes follow")
    args = ap.parse_args()
    wl, g = synth.workload(args.workload), synth.make_graph(args.workload)
    dec = W.Decoder(W.Graph(g, device=0), W.make_params(wl.search_beam, wl.output_beam, wl.min_active, wl.max_active, True),
                    max_lanes=wl.B, max_frames=wl.T)
    lp = torch.from_numpy(synth.make_log_probs(args.workload)).cuda()
    words = [[int(w) for w in r["words"]] for r in dec.decode(lp, synth.make_lens(args.workload))]
    lm = LanguageModel.random(Shape(vocab=int(max(g["olabel"].max(), 0)) + 1))
    longest = max(map(len, words)) + args.new_tokens
    second = SecondPass(lm, max_lanes=len(words), max_tokens=longest,
                        pages=len(words) * -(-longest // 64) + -(-args.prefix // 64))
    second.read_prefix(np.random.default_rng(0).integers(0, lm.shape.vocab, args.prefix))
    second.run(words, args.new_tokens, top_p=args.top_p)
    torch.cuda.synchronize()
    start = time.perf_counter()
    answers = second.run(words, args.new_tokens, top_p=args.top_p)
    spent = time.perf_counter() - start
    for b, (w, a) in enumerate(zip(words, answers)):
        print(f"lane {b}: {len(w)} words {w[:8]}... -> {a['tokens'][:8]}...")
    steps = longest
    for b, w in enumerate(second.score(words)):
        print(f"lane {b}: {sum(w['logprobs']):.2f} for its words")
    print(f"{len(words)} lanes, {steps} steps, {spent / steps * 1e6:.0f} us a step")


if __name__ == "__main__":
    main()
