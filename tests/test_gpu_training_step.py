"""The operators of a training step of adapters beside 8-bit weights, together: the weights' and the input's codes, their
product with lora_add on it, policy_loss in place, lora_grad from the codes and the input's gradient through the
transposed weights; and what single calls of them have to stand."""
import numpy as np
import pytest

from examples import recover_head
from oracle import fp8 as F8
from oracle import grads as F
from tests import answer_data as D
from tests.gpu_run import log
from tests.test_gpu_lora_grad import bounds, check

pytestmark = pytest.mark.gpu
CLIP, KL = 0.2, 0.1


class Step:
    """One step on kept buffers; `refresh` gives other inputs in the same places."""

    def __init__(self, M, d_in, vocab, rank, n):
        import torch
        from post_weight_quantization_08_amd import pipeline as P
        self.sizes = M, d_in, vocab, rank, n
        gen = torch.Generator(device="cuda").manual_seed(11)

        def randn(*shape):
            return torch.randn(*shape, generator=gen, device="cuda")
        self.randn = randn
        self.W = (randn(vocab, d_in) * d_in ** -0.5).bfloat16()
        self.X = randn(M, d_in).bfloat16()
        self.A = (randn(n, rank, d_in) * d_in ** -0.5).bfloat16()
        self.B = (randn(n, vocab, rank) * 0.3).bfloat16()
        self.scale = torch.rand(n, generator=gen, device="cuda") + 0.5
        self.adapter = torch.randint(-1, n, (M,), generator=gen, device="cuda", dtype=torch.int32)
        self.targets = torch.randint(0, vocab, (M,), generator=gen, device="cuda", dtype=torch.int32)
        self.adv = randn(M)
        self.weight = torch.rand(M, generator=gen, device="cuda") / M
        self.old, self.ref = torch.zeros(M, device="cuda"), torch.zeros(M, device="cuda")
        self.head = P.fp8_quantize(self.W, tiles=True)
        self.kept = P.fp8_quantize_buffers(self.X)
        self.base, self.ws_base = P.fp8_matmul_buffers(self.X, self.head["codes"], y_dtype=torch.bfloat16)
        self.logits, self.ws_lora = P.lora_buffers(self.X, self.A, self.B, torch.bfloat16)
        self.loss, self.ws_loss = P.policy_loss_buffers(self.logits, want_grad=False)
        self.loss["grad"] = self.logits
        self.grads, self.ws_grad = P.lora_grad_buffers(self.kept["codes"], self.logits, self.A, self.B, torch.float32)
        _, self.ws_back = P.fp8_matmul_buffers(self.logits, self.head["codes_t"])

    def forward(self):
        from post_weight_quantization_08_amd import pipeline as P
        P.fp8_quantize(self.X, out=self.kept)
        P.fp8_matmul(self.kept["codes"], self.head["codes"], self.head["scales"], x_scales=self.kept["scales"],
                     Y=self.base, ws=self.ws_base)
        P.lora_add(self.X, self.A, self.B, self.adapter, self.scale, base=self.base, Y=self.logits, ws=self.ws_lora)

    def run(self):
        from post_weight_quantization_08_amd import pipeline as P
        self.forward()
        P.policy_loss(self.logits, self.targets, self.old, self.adv, self.ref, CLIP, CLIP, KL, weight=self.weight,
                      out=self.loss, ws=self.ws_loss)
        dx = self.grads["dX"]
        P.fp8_matmul(self.logits, self.head["codes_t"], self.head["scales_t"], Y=dx, ws=self.ws_back)
        P.lora_grad(self.kept["codes"], self.logits, self.A, self.B, self.adapter, self.scale,
                    x_scales=self.kept["scales"], base=dx, out=self.grads, ws=self.ws_grad)

    def behave(self):
        """Log probabilities of a behaviour and a reference near the model: ratios inside the clip's range."""
        import torch
        from post_weight_quantization_08_amd import pipeline as P
        self.forward()
        lp = P.token_logprobs(self.logits, self.targets)["logprob"]
        self.old.copy_(lp + 0.1 * torch.rand_like(lp) - 0.05)
        self.ref.copy_(lp + 0.3 * self.randn(*lp.shape))

    def refresh(self):
        self.X.copy_(self.randn(*self.X.shape))
        self.B.add_(0.1 * self.randn(*self.B.shape))
        self.adapter.copy_(self.adapter.roll(7))
        self.behave()

    def outputs(self):
        out = {"base": self.base, "dlogits": self.logits, **{k: v for k, v in self.loss.items() if k != "grad"}}
        out.update(self.grads)
        return {k: v.clone() for k, v in out.items()}


@pytest.mark.parametrize("M,d_in,vocab,rank,n", [(1, 128, 300, 8, 1), (40, 200, 515, 16, 3), (700, 384, 1000, 64, 2)])
def test_a_step_eager_captured_and_on_other_inputs(M, d_in, vocab, rank, n):
    import torch
    s = Step(M, d_in, vocab, rank, n)
    s.behave()
    s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for r in range(4):
        s.refresh()
        s.run()
        want = s.outputs()
        for t in [s.base, s.logits, *s.grads.values(), *(v for v in s.loss.values())]:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        got = s.outputs()
        for k in want:
            assert torch.equal(want[k], got[k]), (r, k)


@pytest.mark.parametrize("M,d_in,vocab,rank,n", [(40, 200, 515, 16, 3), (300, 384, 260, 40, 2)])
def test_a_step_against_float64(M, d_in, vocab, rank, n):
    """dA, dB and dX from the GPU's own dlogits; and dA, dB against differences of the losses in float64."""
    import torch
    s = Step(M, d_in, vocab, rank, n)
    s.behave()
    s.run()
    torch.cuda.synchronize()

    def f64(t):
        return t.double().cpu().numpy()
    x = F8.fp8_values(s.kept["codes"].view(torch.uint8).cpu().numpy(), s.kept["scales"].view(torch.uint8).cpu().numpy())[:, :d_in]
    w = F8.fp8_values(s.head["codes"].view(torch.uint8).cpu().numpy(), s.head["scales"].view(torch.uint8).cpu().numpy(),
                      tiles=True)[:, :d_in]
    wt = F8.fp8_values(s.head["codes_t"].view(torch.uint8).cpu().numpy(),
                       s.head["scales_t"].view(torch.uint8).cpu().numpy(), tiles=True)[:, :vocab]
    assert np.array_equal(wt.T, w)
    g, A, B, ad, sc = f64(s.logits), f64(s.A), f64(s.B), s.adapter.cpu().numpy(), f64(s.scale)
    # dX: the product of the quantized dlogits, then the adapters'; the product's own error comes with the base
    q = F8.fp8_values(*F8.fp8_quantize(g))[:, :vocab]
    base = q @ w
    want = F.lora_grad(x, g, A, B, ad, sc, base)
    got = {k: f64(s.grads[k]) for k in want}
    b = bounds(x, g, A, B, ad, sc, "bf16", "bf16", want, base, "f32")
    b["dX"] += (np.abs(q) @ np.abs(w)) * 2.0 ** -23 * (vocab + 16)
    check(got, want, b, f"step {M}x{d_in}x{vocab}")

    # losses in float64 from the input itself for the adapters and its codes for the weights
    xx = f64(s.X)
    old, ref, adv, t, wgt = f64(s.old), f64(s.ref), f64(s.adv), s.targets.cpu().numpy(), f64(s.weight)
    rows = np.flatnonzero(ad >= 0)

    def logits(A, B):
        z = x @ w.T
        for m in rows:
            z[m] += sc[ad[m]] * (B[ad[m]] @ (A[ad[m]] @ xx[m]))
        return z

    def total(A, B):
        return float((wgt * F.policy_loss(logits(A, B), t, old, adv, ref, CLIP, CLIP, KL)["loss"]).sum())
    z = logits(A, B)
    o = F.policy_loss(z, t, old, adv, ref, CLIP, CLIP, KL)
    assert (np.abs(o["ratio"] - 1) < 0.15).all()
    # A logit is rounded twice to bf16 (the product, with 8-bit instructions off by 7 2^-13 of a block's largest
    # products, and the sum); a probability moves by twice that, relatively, and so do the ratio and exp(ref - lp)
    z0 = x @ w.T
    dz = (2.0 ** -8 * (np.abs(z0) + np.abs(z)) + 7 * 2.0 ** -13 * (np.abs(x) @ np.abs(w).T)).max(1, keepdims=True)
    e = np.exp(z - z.max(1, keepdims=True))
    p = e / e.sum(1, keepdims=True)
    hot = np.zeros_like(p)
    hot[np.arange(M), t] = 1
    move = 2 * dz * np.exp(2 * dz)
    size = ((np.abs(adv) * o["ratio"] + KL * np.exp(ref - o["logprob"]) + KL) * wgt)[:, None]
    dg = size * (p + hot) * (2 * move) + np.abs(g) * 2.0 ** -8 + 1e-9
    # A's gradient is taken at the codes of the input: the exact one there differs by what quantization moved it
    for k, at in (("dA", 0), ("dB", 1)):
        d = got[k] / np.linalg.norm(got[k])
        h = 1e-5
        ends = [total(*[v + sign * h * d if i == at else v for i, v in enumerate((A, B))]) for sign in (1, -1)]
        slack, moved = 0.0, 0.0
        for m in rows:
            a = ad[m]
            if k == "dA":
                j, je = B[a] @ (d[a] @ xx[m]), B[a] @ (d[a] @ (x[m] - xx[m]))
            else:
                j, je = d[a] @ (A[a] @ xx[m]), d[a] @ (A[a] @ (x[m] - xx[m]))
            slack += sc[a] * (np.abs(j) + np.abs(je)) @ dg[m]
            moved += sc[a] * (g[m] @ je)
        num = (ends[0] - ends[1]) / (2 * h)
        err = abs((got[k] * d).sum() - moved - num)
        log(f"[gpu] step {M}x{d_in}x{vocab} {k}: by differences {num:.6f}, off {err:.1e} of {slack:.1e}")
        assert err <= slack + 1e-5 * abs(num)


def test_the_example_s_gradients():
    import torch
    from post_weight_quantization_08_amd import pipeline as P
    gen = torch.Generator(device="cuda").manual_seed(5)
    M, d_in, vocab, rank, n = 130, 256, 601, 16, 2
    X = torch.randn(M, d_in, generator=gen, device="cuda").bfloat16()
    A = (torch.randn(n, rank, d_in, generator=gen, device="cuda") * d_in ** -0.5).bfloat16()
    B = torch.randn(n, vocab, rank, generator=gen, device="cuda").bfloat16()
    g = (torch.randn(M, vocab, generator=gen, device="cuda") / M).bfloat16()
    ad = (torch.arange(M, device="cuda") * 2 // M).int()
    scale = torch.tensor([1.0, 0.5], device="cuda")
    kept = P.fp8_quantize(X)
    dA, dB = recover_head.gradients(kept, A, B, ad, scale, g)
    x = F8.fp8_values(kept["codes"].view(torch.uint8).cpu().numpy(), kept["scales"].view(torch.uint8).cpu().numpy())
    args = [x, *(t.double().cpu().numpy() for t in (g, A, B))]
    want = {k: v for k, v in F.lora_grad(*args, ad.cpu().numpy(), scale.double().cpu().numpy()).items() if k != "dX"}
    b = bounds(*args, ad.cpu().numpy(), scale.double().cpu().numpy(), "bf16", "bf16", want, None, None)
    check({"dA": dA.double().cpu().numpy(), "dB": dB.double().cpu().numpy()}, want, b, "example")


def test_the_last_row_of_b_stays_in_its_column():
    """An infinity in B's last row gives infinities in U's column of its rank and nothing elsewhere, whether d_out ends
    inside a block or not."""
    import torch
    from post_weight_quantization_08_amd import pipeline as P
    for d_out, rank in ((130, 8), (130, 33), (256, 8)):
        X = torch.ones(20, 64, device="cuda").bfloat16()
        A = torch.ones(1, rank, 64, device="cuda").bfloat16()
        B = torch.ones(1, d_out, rank, device="cuda").bfloat16()
        B[0, -1, 0] = float("inf")
        g = torch.ones(20, d_out, device="cuda").bfloat16()
        ad = torch.zeros(20, dtype=torch.int32, device="cuda")
        out = P.lora_grad(X, g, A, B, ad)
        assert torch.isposinf(out["dA"][0, 0]).all(), (d_out, rank)
        assert (out["dA"][0, 1:] == 20 * d_out).all() and (out["dB"] == 20 * 64).all()


@pytest.mark.parametrize("M,n", [(64, 3), (640, 4), (32, 1000)])
def test_nothing_stands_where_the_last_adapters_have_no_tokens(M, n):
    import torch
    from post_weight_quantization_08_amd import pipeline as P
    gen = torch.Generator(device="cuda").manual_seed(6)
    X, g = (torch.randn(M, w, generator=gen, device="cuda").bfloat16() for w in (200, 300))
    A, B = torch.randn(n, 8, 200, device="cuda").bfloat16(), torch.randn(n, 300, 8, device="cuda").bfloat16()
    ad = torch.zeros(M, dtype=torch.int32, device="cuda")
    out, ws = P.lora_grad_buffers(X, g, A, B, torch.bfloat16)
    one = P.lora_grad(X, g, A[:1].contiguous(), B[:1].contiguous(), ad, want_dx=True)
    ws.fill_(0x7F)
    P.lora_grad(X, g, A, B, ad, out=out, ws=ws)
    assert not out["dA"][1:].any() and not out["dB"][1:].any()
    for k in ("dA", "dB"):
        assert torch.equal(out[k][:1], one[k]), k
    assert torch.equal(out["dX"], one["dX"])


def test_a_wanted_dx_needs_a_place():
    import torch
    from post_weight_quantization_08_amd import pipeline as P
    X, g = torch.zeros(4, 64, device="cuda").bfloat16(), torch.zeros(4, 32, device="cuda").bfloat16()
    A, B = torch.zeros(1, 8, 64, device="cuda").bfloat16(), torch.zeros(1, 32, 8, device="cuda").bfloat16()
    out, ws = P.lora_grad_buffers(X, g, A, B)
    ad = torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="want_dx"):
        P.lora_grad(X, g, A, B, ad, want_dx=True, out=out, ws=ws)
    assert "dX" not in P.lora_grad(X, g, A, B, ad, out=out, ws=ws)
