"""Quantise a small routed layer and serve it from its packed words.

A projection with low-rank adapters of several requests beside it, then a router over experts with a gated activation:
the weights go through the library's quantisation (Gram, factor, column loop, packing), the tokens through its serving
calls, once as ragged prompts and once as single tokens.  Prints how far the results are from the same codes in float64.

    python examples/serve_layer.py [--experts 4] [--features 512] [--inner 768] [--bits 4] [--groupsize 128]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import post_weight_quantization_09_amd as G  # noqa: E402

DEV = "cuda"


def quantised(K, N, bits, groupsize, gen):
    """A random layer, calibrated and quantised: its packed words, its scales and its weights in float64."""
    W = torch.randn(K, N, generator=gen, device=DEV) * 0.05
    X = torch.randn(4 * K, K, generator=gen, device=DEV).to(torch.bfloat16)
    H = torch.zeros(K, K, device=DEV)
    G.gptq_accumulate_hessian(H, X)
    dead, _, _ = G.gptq_prepare(H, 0.01)
    q = G.gptq_quantize_layer(W, H, bits, dead=dead, groupsize=groupsize)
    s = q["scales"].double()
    s = s.repeat_interleave(groupsize, 0)[:K] if groupsize else s
    return G.gptq_pack_codes(q["codes"], bits), q["scales"], s * (q["codes"].double() - 2 ** (bits - 1))


class RoutedLayer:
    def __init__(self, a, gen):
        self.bits, self.groupsize, self.topk = a.bits, a.groupsize, 2
        self.proj = quantised(a.features, a.features, a.bits, a.groupsize, gen)
        up = [quantised(a.features, 2 * a.inner, a.bits, a.groupsize, gen) for _ in range(a.experts)]
        down = [quantised(a.inner, a.features, a.bits, a.groupsize, gen) for _ in range(a.experts)]
        # words and scales of all experts in one tensor each, laid out once
        self.up, self.down = ((torch.stack([e[0] for e in es]), torch.stack([e[1] for e in es]),
                               [e[2] for e in es]) for es in (up, down))
        self.gate = torch.randn(a.features, a.experts, generator=gen, device=DEV) * 0.2
        self.A = (torch.randn(3, 16, a.features, generator=gen, device=DEV) * 0.05).to(torch.bfloat16)
        self.B = (torch.randn(3, a.features, 16, generator=gen, device=DEV) * 0.05).to(torch.bfloat16)
        self.alpha = torch.tensor([1.0, 0.5, 2.0], device=DEV)

    def forward(self, x, requests, adapter):
        kw = dict(groupsize=self.groupsize)
        h = G.gptq_adapter_matmul(x, self.proj[0], self.proj[1], self.bits, A=self.A, B=self.B, alpha=self.alpha,
                                  requests=requests, adapter=adapter, **kw)
        r = G.gptq_route(h.float() @ self.gate, self.topk, renorm=True)
        u = G.gptq_expert_matmul(h, self.up[0], self.up[1], r["offsets"], self.bits, rows=r["rows"], swiglu=True, **kw)
        y = G.gptq_expert_matmul(u, self.down[0], self.down[1], r["offsets"], self.bits, **kw)
        return h, r, G.gptq_combine(y, r["positions"], r["weights"])

    def check(self, x, requests, adapter, h, r, out):
        """2-norms of the errors of the projection and of the layer behind it, against the same codes in float64."""
        want = x.double() @ self.proj[2]
        for i, a in enumerate(adapter.tolist()):
            if a >= 0:
                rows = slice(int(requests[i]), int(requests[i + 1]))
                want[rows] += self.alpha[a].double() * (x[rows].double() @ self.A[a].double().t()) @ self.B[a].double().t()
        whole = torch.zeros_like(want)
        for e in range(len(self.up[2])):
            t, j = torch.nonzero(r["experts"] == e, as_tuple=True)
            g, u = (h[t].double() @ self.up[2][e]).chunk(2, 1)
            whole.index_add_(0, t, r["weights"][t, j].double()[:, None] * ((g * torch.sigmoid(g) * u) @ self.down[2][e]))
        return [((p.double() - q).norm() / q.norm()).item() for p, q in ((h, want), (out, whole))]


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("experts", 4), ("features", 512), ("inner", 768), ("bits", 4), ("groupsize", 128)):
        p.add_argument("--" + name, type=int, default=default)
    a = p.parse_args()
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    layer = RoutedLayer(a, gen)
    for name, lengths in (("prompts", [37, 200, 1, 90]), ("single tokens", [1, 1, 1, 1])):
        ends = [0]
        for n in lengths:
            ends.append(ends[-1] + n)
        requests = torch.tensor(ends, dtype=torch.int32, device=DEV)
        adapter = torch.tensor([0, 2, -1, 1], dtype=torch.int32, device=DEV)
        x = torch.randn(ends[-1], a.features, generator=gen, device=DEV).to(torch.bfloat16)
        h, r, out = layer.forward(x, requests, adapter)
        errors = layer.check(x, requests, adapter, h, r, out)
        rows = (r["offsets"][1:] - r["offsets"][:-1]).tolist()
        print(f"{name}: {ends[-1]} tokens, rows per expert {rows}, error of the projection {errors[0]:.2e}, "
              f"of the routed layer {errors[1]:.2e}", flush=True)
        assert max(errors) < 1e-2
    print("ok", flush=True)


if __name__ == "__main__":
    main()
