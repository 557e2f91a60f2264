"""Cases of the 8-bit projection's operators, the norm in front of it and the adapters' update, with their plain forms.

Operators:
  rms_fwd   H = X + R, Y = H rstd gamma with rstd = (mean H^2 + eps)^(-1/2): root-mean-square norm with the residual's
            addition; Y in the input's type, in 8-bit floating point with a power-of-two scale per 128 columns, or both
  rms_bwd   its gradients dX (equal to the residual's) and dgamma; the gradient that reaches H past the norm is added
  enc       a matrix in 8-bit floating point with a power-of-two scale for each block of 128 columns of a row, or of
            128 x 128; also its transpose, coded along the other axis
  mm        A B^T of two such matrices: a projection, its input gradient (B the weight's transpose) and its weight
            gradient (both coded along the tokens)
  orth      an adapter update orthogonalised by five Newton-Schulz steps X <- a X + (b X X^T + c (X X^T)^2) X

With ``own`` false ``run`` computes them in elementary torch operations in 32 bits (the Newton-Schulz steps, which
multiply what the first product rounds by several hundred, in 64); with ``own`` true it calls sparse_rank_adapter_amd.
"""
import math

import torch

own = False

BLOCK = 128  # columns that share a scale
KINDS = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
NS = (3.4445, -4.7750, 2.0315)  # a, b, c of a Newton-Schulz step
STEPS, NS_EPS = 5, 1e-7


# ------------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # the norm of a few tokens with the residual's addition: one decode step (OPT-350M hidden size)
        dict(name="rms_fwd_decode", op="rms_fwd", T=17, H=1024, dtype="bf16", residual=True, out="y"),
        # the norm of a training batch ahead of an 8-bit projection with adapters, which read Y as well (OPT-13B)
        dict(name="rms_fwd_fp8_13b", op="rms_fwd", T=8192, H=5120, dtype="bf16", residual=True, out="both"),
        # backward of a small fp32 batch with an odd token count (OPT-350M)
        dict(name="rms_bwd_350m", op="rms_bwd", T=333, H=1024, dtype="f32", residual=False),
        # backward of a training batch, the residual's own gradient added (OPT-13B)
        dict(name="rms_bwd_13b", op="rms_bwd", T=8191, H=5120, dtype="bf16", residual=True),
        # an output gradient coded for both products of the backward, odd token count (OPT-350M fc1)
        dict(name="enc_grad_350m", op="enc", R=2047, C=4096, dtype="bf16", kind="e5m2", rows=1, form="pair"),
        # a weight and its transpose coded in 128 x 128 blocks after an update (OPT-13B fc1)
        dict(name="enc_weight_13b", op="enc", R=20480, C=5120, dtype="bf16", kind="e4m3", rows=128, form="pair"),
        # one decode step of 16 requests over the OPT-66B FFN weight
        dict(name="mm_decode_66b", op="mm", M=16, K=9216, N=36864, a="e4m3", b="e4m3", rows=128, out="bf16"),
        # a prompt batch (OPT-13B fc1)
        dict(name="mm_prompt_13b", op="mm", M=8192, K=5120, N=20480, a="e4m3", b="e4m3", rows=128, out="bf16"),
        # input gradient: dY in e5m2 against the weight's transpose, odd token count (OPT-350M fc1)
        dict(name="mm_dx_350m", op="mm", M=2047, K=4096, N=1024, a="e5m2", b="e4m3", rows=128, out="bf16"),
        # weight gradient: both operands coded along an odd number of tokens (OPT-350M fc1)
        dict(name="mm_dw_350m", op="mm", M=4096, K=2047, N=1024, a="e5m2", b="e4m3", rows=1, out="f32"),
        # the updates of a dozen small adapters, A [16, 1024] each (OPT-350M fc1)
        dict(name="orth_a_350m", op="orth", n=12, R=16, C=1024, dtype="f32"),
        # the updates of eight large adapters, B [20480, 128] each (OPT-13B fc1)
        dict(name="orth_b_13b", op="orth", n=8, R=20480, C=128, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rms_fwd", "rms_bwd", "enc", "mm", "mm", "orth"])
    dtype = rng.choice(["bf16", "f32"])
    if op in ("rms_fwd", "rms_bwd"):
        H = _log(rng, 65, 12288)
        c = dict(op=op, T=_log(rng, 1, min(8192, 40_000_000 // H)), H=H, dtype=dtype, residual=rng.random() < 0.6)
        if op == "rms_fwd":
            c["out"] = rng.choice(["y", "fp8", "both"])
        return c
    if op == "enc":
        R = _log(rng, 1, 8192)
        return dict(op=op, R=R, C=_log(rng, 33, min(20480, 50_000_000 // R)), dtype=dtype,
                    kind=rng.choice(["e4m3", "e5m2"]), rows=rng.choice([1, 128]), form=rng.choice(["rows", "pair"]))
    if op == "mm":
        M = _log(rng, 1, 64) if rng.random() < 0.3 else _log(rng, 65, 8192)
        return dict(op=op, M=M, K=_log(rng, 100, 9216), N=_log(rng, 100, 9216), a=rng.choice(["e4m3", "e5m2"]),
                    b="e4m3", rows=rng.choice([1, 128]), out=rng.choice(["bf16", "f32"]))
    d, n = _log(rng, 4, 256), _log(rng, 1, 16)
    L = _log(rng, d, max(d, min(8192, 2_500_000_000 // (n * d * d))))
    R, C = rng.choice([(d, L), (L, d)])
    return dict(op=op, n=n, R=R, C=C, dtype=dtype)


# ------------------------------------------------------------------------------------------ inputs
def _dt(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _normal(g, *shape, sd=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device="cuda") * sd).to(dtype)


def _activations(g, T, K, dtype=torch.bfloat16):
    """Unit normal columns with a few loud channels, as the inputs of a projection have."""
    loud = torch.where(torch.rand(K, generator=g, device="cuda") < 0.01, 12.0, 1.0)
    return (torch.randn(T, K, generator=g, device="cuda") * loud).to(dtype)


def _gradients(g, T, N, dtype=torch.bfloat16):
    """Output gradients: small, and of very different sizes from token to token."""
    size = 1e-4 * torch.exp(1.5 * torch.randn(T, 1, generator=g, device="cuda"))
    return (torch.randn(T, N, generator=g, device="cuda") * size).to(dtype)


def _operand(g, rows, cols, kind, block_rows, grad=False, sd=1.0):
    """A matrix as a program keeps it: codes with their rows filled up to whole blocks, and scale exponents."""
    codes, exps = [], []
    for lo in range(0, rows, 4096):
        n = min(4096, rows - lo)
        x = _gradients(g, n, cols) if grad else _activations(g, n, cols) * sd
        c, e = _encode(x, kind, block_rows)
        codes.append(c)
        exps.append(e)
    return dict(codes=torch.cat(codes), exps=torch.cat(exps), rows=rows, cols=cols, block_rows=block_rows)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    if op in ("rms_fwd", "rms_bwd"):
        T, H, dt = case["T"], case["H"], _dt(case["dtype"])
        s["X"], s["gamma"], s["eps"] = _activations(g, T, H, dt), _normal(g, H, sd=0.1, dtype=dt) + 1, 1e-6
        if op == "rms_fwd":
            s["R"] = _activations(g, T, H, dt) if case["residual"] else None
        else:
            s["dY"], s["dH"] = _gradients(g, T, H, dt), _gradients(g, T, H, dt) if case["residual"] else None
            s["rstd"] = torch.rsqrt(s["X"].float().square().mean(1) + s["eps"])
    elif op == "enc":
        make = _gradients if case["kind"] == "e5m2" else _activations
        s["X"] = make(g, case["R"], case["C"], _dt(case["dtype"]))
    elif op == "mm":
        s["A"] = _operand(g, case["M"], case["K"], case["a"], 1, grad=case["a"] == "e5m2")
        s["B"] = _operand(g, case["N"], case["K"], case["b"], case["rows"], sd=0.02)
    else:
        n, R, C = case["n"], case["R"], case["C"]
        k = min(R, C, 24)  # a gradient has some strong directions, and noise in all of them
        size = torch.logspace(0, -2, k, device="cuda")
        low = torch.randn(n, R, k, generator=g, device="cuda") * size
        G = torch.bmm(low, torch.randn(n, k, C, generator=g, device="cuda"))
        s["G"] = (1e-3 * (G + 0.01 * torch.randn(n, R, C, generator=g, device="cuda"))).to(_dt(case["dtype"]))
    return s


# ------------------------------------------------------------------------------------------ plain forms, 32 bits
def _pow2(e):
    return ((e + 127) << 23).view(torch.float32)


def _encode(X, kind, block_rows):
    """Codes [R, C rounded up to whole blocks] and exponents uint8 [ceil(R / block_rows), ceil(C / 128)] (2^(e - 127)):
    the smallest power of two with every |x| of the block at most 448 (e5m2: 57344) times it."""
    R, C = X.shape
    top, most = (8, 119) if kind == "e4m3" else (15, 112)  # 448 = 1.75 2^8, 57344 = 1.75 2^15
    x = torch.nn.functional.pad(X.float(), (0, -C % BLOCK, 0, -R % block_rows))
    x = x.reshape(-1, block_rows, x.shape[1] // BLOCK, BLOCK)
    m, ex = torch.frexp(x.abs().amax((1, 3)))
    e = torch.where(m == 0, -126, ex.int() - 1 - top + (m > 0.875).int()).clamp(-126, most).int()
    lim = 1.75 * 2.0 ** top
    q = (x * _pow2(-e)[:, None, :, None]).clamp(-lim, lim).to(KINDS[kind])
    return q.reshape(x.shape[0] * block_rows, -1)[:R].contiguous(), (e + 127).to(torch.uint8)


def _decode(codes, exps, cols, block_rows):
    s = _pow2(exps.int() - 127).repeat_interleave(block_rows, 0)[:codes.shape[0]]
    return (codes.float() * s.repeat_interleave(BLOCK, 1))[:, :cols]


def _values(F):
    return _decode(F["codes"], F["exps"], F["cols"], F["block_rows"])


def _coded(X, kind, block_rows):
    """The values that X's codes stand for."""
    return _decode(*_encode(X, kind, block_rows), X.shape[1], block_rows)


def _ns_step(X):
    a, b, c = NS
    A = torch.bmm(X, X.transpose(1, 2).contiguous())
    return a * X + torch.bmm(b * A + c * torch.bmm(A, A), X)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "rms_fwd":
        x = s["X"].float()
        h = x if s["R"] is None else x + s["R"].float()
        rstd = torch.rsqrt(h.square().mean(1) + s["eps"])
        y = h * rstd[:, None] * s["gamma"].float()
        out = dict(rstd=rstd)
        if s["R"] is not None:
            out["H"] = h.to(s["X"].dtype)
        if case["out"] != "fp8":
            out["Y"] = y.to(s["X"].dtype)
        if case["out"] != "y":
            out["coded"] = _coded(y, "e4m3", 1).bfloat16()
        return out
    if op == "rms_bwd":
        dy, rstd = s["dY"].float(), s["rstd"][:, None]
        xh = s["X"].float() * rstd
        gy = dy * s["gamma"].float()
        dx = rstd * (gy - xh * (gy * xh).mean(1, keepdim=True))
        if s["dH"] is not None:
            dx = dx + s["dH"].float()
        return dict(dX=dx.to(s["X"].dtype), dgamma=(dy * xh).sum(0))
    if op == "enc":
        out = dict(coded=_coded(s["X"], case["kind"], case["rows"]).bfloat16())
        if case["form"] == "pair":
            out["coded_t"] = _coded(s["X"].t().contiguous(), case["kind"], case["rows"]).bfloat16()
        return out
    if op == "mm":
        return dict(Y=(_values(s["A"]) @ _values(s["B"]).t()).to(_dt(case["out"])))
    wide = case["R"] <= case["C"]
    X = s["G"].double() if wide else s["G"].double().transpose(1, 2).contiguous()
    X = X / (X.square().sum((1, 2), keepdim=True).sqrt() + NS_EPS)
    X = _ns_step(_ns_step(_ns_step(_ns_step(_ns_step(X)))))
    return dict(O=(X if wide else X.transpose(1, 2)).to(s["G"].dtype).contiguous())


# ------------------------------------------------------------------------------------------ the framework's calls
def _own(s):
    import sparse_rank_adapter_amd as sra
    case = s["case"]
    op = case["op"]

    def matrix(F):
        return sra.Fp8Matrix(F["codes"], F["exps"], F["rows"], F["cols"], F["block_rows"])

    if op == "rms_fwd":
        fp8 = None if case["out"] == "y" else torch.float8_e4m3fn
        Y, H, rstd, c = sra.rms_norm_fwd(s["X"], s["gamma"], s["eps"], residual=s["R"], fp8=fp8,
                                         want_y=case["out"] != "fp8")
        out = dict(rstd=rstd)
        if s["R"] is not None:
            out["H"] = H
        if case["out"] != "fp8":
            out["Y"] = Y
        if fp8 is not None:
            out["coded"] = sra.fp8_decode(c)
        return out
    if op == "rms_bwd":
        dX, dgamma = sra.rms_norm_bwd(s["dY"], s["X"], s["gamma"], s["rstd"], dH=s["dH"])
        return dict(dX=dX, dgamma=dgamma)
    if op == "enc":
        if case["form"] == "pair":
            c, ct = sra.fp8_encode_pair(s["X"], KINDS[case["kind"]], block_rows=case["rows"])
            return dict(coded=sra.fp8_decode(c), coded_t=sra.fp8_decode(ct))
        return dict(coded=sra.fp8_decode(sra.fp8_encode(s["X"], KINDS[case["kind"]], block_rows=case["rows"])))
    if op == "mm":
        return dict(Y=sra.fp8_matmul(matrix(s["A"]), matrix(s["B"]), out_dtype=_dt(case["out"])))
    return dict(O=sra.orthogonalize(s["G"], steps=STEPS, coeffs=NS, eps=NS_EPS))


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ------------------------------------------------------------------------------------------ floors
def _size(name):
    return 4 if name == "f32" else 2


def work(case):
    op = case["op"]
    if op in ("rms_fwd", "rms_bwd"):
        T, H, e = case["T"], case["H"], _size(case["dtype"])
        if op == "rms_fwd":
            n = T * H * e * (3 if case["residual"] else 1) + H * e + 4 * T
            n += 0 if case["out"] == "fp8" else T * H * e
            n += 0 if case["out"] == "y" else 2 * T * H  # the values the codes stand for
            return dict(bytes=n, flops=5 * T * H)
        return dict(bytes=T * H * e * (4 if case["residual"] else 3) + H * e + 4 * H + 4 * T, flops=10 * T * H)
    if op == "enc":
        n = case["R"] * case["C"]
        forms = 2 if case["form"] == "pair" else 1
        return dict(bytes=n * (_size(case["dtype"]) + 2 * forms), flops=3 * n * forms)
    if op == "mm":
        M, K, N = case["M"], case["K"], case["N"]
        scales = -(-K // BLOCK) * (M + -(-N // case["rows"]))
        return dict(bytes=(M + N) * K + scales + M * N * _size(case["out"]), flops=2 * M * N * K)
    d, L = sorted((case["R"], case["C"]))
    # one symmetric product of the update with itself and one product with the d x d result
    return dict(bytes=2 * case["n"] * d * L * _size(case["dtype"]), flops=case["n"] * d * (d + 1 + 2 * d) * L)


# ------------------------------------------------------------------------------------------ 64 bits
def _two(k):
    return ((k.long() + 1023) << 52).view(torch.float64)


def _coded64(X, kind, block_rows):
    """Values of X after 8-bit coding, in 64 bits: each block over the power of two that brings it under the type's
    largest value, rounded to the type's steps (3 or 2 bits below the leading one, and no finer than its smallest)."""
    R, C = X.shape
    bits, low, lim, most = (3, -6, 448.0, 119) if kind == "e4m3" else (2, -14, 57344.0, 112)
    p = torch.zeros(-(-R // block_rows) * block_rows, -(-C // BLOCK) * BLOCK, dtype=torch.float64, device=X.device)
    p[:R, :C] = X.double()
    p = p.view(-1, block_rows, p.shape[1] // BLOCK, BLOCK)
    top = p.abs().amax(3).amax(1)[:, None, :, None]
    e = torch.full_like(top, -126.0)
    live = top > 0
    e[live] = torch.ceil(torch.log2(top[live] / lim))
    e = e.clamp(-126, most)
    e = torch.where(live & (top > lim * _two(e)) & (e < most), e + 1, e)  # log2's rounding at the border
    e = torch.where(live & (e > -126) & (top <= lim * _two(e - 1)), e - 1, e)
    v = p * _two(-e)
    step = _two(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** low))).clamp(low, 20) - bits)
    q = (torch.round(v / step) * step).clamp(-lim, lim) * _two(e)
    return q.reshape(-1, q.shape[2] * BLOCK)[:R, :C]


def _values64(F):
    e = F["exps"].long().repeat_interleave(F["block_rows"], 0)[:F["rows"]].repeat_interleave(BLOCK, 1)
    return (F["codes"].double() * _two(e - 127))[:, :F["cols"]]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rms_fwd":
        h = s["X"].double()
        out = dict()
        if s["R"] is not None:
            h = h + s["R"].double()
        rstd = 1 / torch.sqrt((h * h).sum(1) / case["H"] + s["eps"])
        y = h * s["gamma"].double() * rstd[:, None]
        out["rstd"] = rstd
        if s["R"] is not None:
            out["H"] = h
        if case["out"] != "fp8":
            out["Y"] = y
        if case["out"] != "y":
            out["coded"] = _coded64(y, "e4m3", 1)
        return out
    if op == "rms_bwd":
        x, dy, rstd = s["X"].double(), s["dY"].double(), s["rstd"].double()[:, None]
        gy = dy * s["gamma"].double()
        dX = rstd * gy - x * rstd ** 3 * ((gy * x).sum(1, keepdim=True) / case["H"])
        if s["dH"] is not None:
            dX += s["dH"].double()
        return dict(dX=dX, dgamma=(dy * x * rstd).sum(0))
    if op == "enc":
        out = dict(coded=_coded64(s["X"], case["kind"], case["rows"]))
        if case["form"] == "pair":
            out["coded_t"] = _coded64(s["X"].t(), case["kind"], case["rows"])
        return out
    if op == "mm":
        return dict(Y=_values64(s["A"]) @ _values64(s["B"]).t())
    # by the singular values: every step maps a value v to a v + b v^3 + c v^5 and leaves the vectors
    G = s["G"].double()
    tall = case["R"] > case["C"]
    lam, V = torch.linalg.eigh((G.mT.contiguous() @ G) if tall else (G @ G.mT.contiguous()))
    lam = lam.clamp(min=0)
    norm = lam.sum(1, keepdim=True).sqrt() + NS_EPS
    v = lam.sqrt() / norm
    gain = torch.ones_like(v)
    for _ in range(STEPS):
        f = NS[0] + NS[1] * v ** 2 + NS[2] * v ** 4
        v, gain = v * f, gain * f
    Q = (V * (gain / norm)[:, None, :]) @ V.mT.contiguous()
    return dict(O=G @ Q if tall else Q @ G)
