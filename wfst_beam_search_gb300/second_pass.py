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

``python -m wfst_beam_search_gb300.second_pass`` (in the source tree) decodes a
synthetic workload and runs such a pass, with random weights, on its words.
"""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np
import torch
import torch.nn.functional as F

from . import _ops


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
        self.device = self.embed.device    # with its number, whatever is the current device later
        self.layers = [{name: take(f"{i}.{name}") for name in
                        ("gain1", "qkv", "q_gain", "k_gain", "out", "gain2", "up", "down")} for i in range(s.layers)]

    @classmethod
    def random(cls, shape, seed=0, dtype=torch.bfloat16, device="cuda"):
        return cls(shape, random_tensors(shape, seed), dtype, device)


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
    one pool of ``pages`` (by default enough for all lanes at full length)."""

    def __init__(self, model, max_lanes, max_tokens, page_size=64, pages=None):
        s, dev = model.shape, model.device
        self.model, self.lanes, self.max_tokens, self.page = model, max_lanes, max_tokens, page_size
        per_lane = -(-max_tokens // page_size)
        self.pages = max_lanes * per_lane if pages is None else pages
        self.cache = [torch.zeros(2, self.pages, page_size, s.kv_heads, s.head_dim, dtype=model.dtype, device=dev)
                      for _ in range(s.layers)]
        self.table = torch.zeros(max_lanes, per_lane, dtype=torch.int32, device=dev)
        angle = (torch.arange(max_tokens, dtype=torch.float64)[:, None]
                 * s.base ** (-torch.arange(0, s.head_dim, 2, dtype=torch.float64) / s.head_dim))
        self.rotary = torch.cat([angle.cos(), angle.sin()], 1).float().to(dev)
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

    def logits(self, tokens, positions, slots, lengths):
        """One token per lane through the model; its keys and values are put
        into the cache.  int32 [lanes] each; a lane with slot -1 and length 0
        is idle."""
        m, s, lanes = self.model, self.model.shape, tokens.shape[0]
        hq, hkv = s.q_heads, s.kv_heads
        x = F.embedding(tokens, m.embed)
        for layer, (keys, values) in zip(m.layers, self.cache):
            h = _ops.matvec_quant(F.rms_norm(x, (s.width,), layer["gain1"], s.eps), layer["qkv"])
            h = h.view(lanes, hq + 2 * hkv, s.head_dim)
            q = _ops.norm_rotate(h[:, :hq], h[:, hq:hq + hkv], h[:, hq + hkv:], positions, self.rotary,
                                 layer["q_gain"], layer["k_gain"], keys, values, slots, eps=s.eps)
            o = _ops.attend_paged(q, keys, values, self.table, lengths, window=s.window, sinks=s.sinks,
                                  workspace=self.workspace)
            x = x + _ops.matvec_quant(o.view(lanes, -1), layer["out"])
            h = _ops.matvec_quant(F.rms_norm(x, (s.width,), layer["gain2"], s.eps), layer["up"])
            x = x + _ops.matvec_quant(F.silu(h[:, :s.hidden]) * h[:, s.hidden:], layer["down"])
        return _ops.matvec_quant(F.rms_norm(x, (s.width,), m.gain, s.eps), m.head)

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
        self.graph = graph

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
        if sum(need) > self.pages:
            raise ValueError(f"the lanes take {sum(need)} pages, the pool has {self.pages}")
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
            plan[:n, 1, b] = at
            plan[:n, 2, b] = table[b, at // self.page] * self.page + at % self.page
            plan[:n, 3, b] = at + 1
        return plan, table

    def run(self, words, new_tokens, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, seed=0, graph=True):
        """Read each lane's ``words`` and draw ``new_tokens`` tokens after
        them: [{"tokens", "logprobs"}, ...].  The same seed draws the same.
        An answer ends where its logits hold no number (weights or activations
        that left the type's range): tokens -1, logprobs -inf from there on."""
        # (``sample_tokens`` refuses numbers, but here they reach it as a value per lane)
        for name, fits in (("temperature", 0 <= temperature <= 3e38), ("top_k", 0 <= top_k < 2 ** 31), ("top_p", top_p > 0),
                           ("min_p", 0 <= min_p <= 1)):
            if not fits:
                raise ValueError(f"{name} is out of range")
        plan, table = self.plan_lanes(words, new_tokens)
        if not len(plan):
            return []
        with torch.cuda.device(self.model.device):    # streams, capture and replay are of the current device
            if graph and self.graph is None:
                self._capture()
            self._load(plan)
            self.table.copy_(torch.from_numpy(table))
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
    args = ap.parse_args()
    wl, g = synth.workload(args.workload), synth.make_graph(args.workload)
    dec = W.Decoder(W.Graph(g, device=0), W.make_params(wl.search_beam, wl.output_beam, wl.min_active, wl.max_active, True),
                    max_lanes=wl.B, max_frames=wl.T)
    lp = torch.from_numpy(synth.make_log_probs(args.workload)).cuda()
    words = [[int(w) for w in r["words"]] for r in dec.decode(lp, synth.make_lens(args.workload))]
    lm = LanguageModel.random(Shape(vocab=int(max(g["olabel"].max(), 0)) + 1))
    second = SecondPass(lm, max_lanes=len(words), max_tokens=max(map(len, words)) + args.new_tokens)
    second.run(words, args.new_tokens, top_p=args.top_p)
    torch.cuda.synchronize()
    start = time.perf_counter()
    answers = second.run(words, args.new_tokens, top_p=args.top_p)
    spent = time.perf_counter() - start
    for b, (w, a) in enumerate(zip(words, answers)):
        print(f"lane {b}: {len(w)} words {w[:8]}... -> {a['tokens'][:8]}...")
    steps = max(map(len, words)) + args.new_tokens
    print(f"{len(words)} lanes, {steps} steps, {spent / steps * 1e6:.0f} us a step")


if __name__ == "__main__":
    main()
