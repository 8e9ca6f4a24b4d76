"""The 8-bit operators of the MLP block, case by case: inputs, plain forms, the framework's calls, work.

Operators (fmax = 448 for e4m3, 57344 for e5m2; a block's scale is max(amax, 2^-100) / fmax and its
values are x * (fmax / max(amax, 2^-100)) rounded to the nearest 8-bit number):

  gemm     C = op(A) op(B)^T over 8-bit operands; A has a scale per row and 128 of the reduction, B
           one per 128 x 128 block (weights) or, for weight gradients, one per column and 128
  rmsnorm  H = X + R, r = rsqrt(mean H^2 + eps), H r g in 8 bits with a scale per row and 128 columns;
           and its backward
  swiglu   the gate/up product with SwiGLU: Y in 8 bits, and [a | b] kept in 8 bits for the backward,
           which reads them and writes the 8-bit operands of the products that follow
  quant    bf16 to 8 bits: rows and columns of an activation's gradient in one pass, or a weight's blocks
"""

import math

import torch

own = False

TINY = 2.0 ** -100
TYPES = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}


def _cdiv(a, b):
    return -(-a // b)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # The down projection of the 7B block's forward on a full batch of tokens.
        {"name": "gemm_down_7B", "op": "gemm", "dir": "fwd", "M": 8192, "N": 4096, "K": 11008, "type": "e4m3"},
        # The gate/up product's input gradient of the 1B block on a ragged batch: the stacked weight is
        # read as it is stored (its rows are the reduction); the gradient is e5m2.
        {"name": "gemm_dgrad_1B_ragged", "op": "gemm", "dir": "dgrad", "M": 1001, "N": 2048, "K": 16384,
         "type": "e5m2"},
        # A weight gradient of the 7B block in fp32 for the master weights, over an odd number of tokens.
        {"name": "gemm_wgrad_7B_odd", "op": "gemm", "dir": "wgrad", "M": 4096, "N": 4096, "K": 8191,
         "type": "e4m3"},
        # One decoding step of three sequences through a square projection: latency counts.
        {"name": "gemm_decode", "op": "gemm", "dir": "fwd", "M": 3, "N": 4096, "K": 4096, "type": "e4m3"},
        # The norm in front of the 7B MLP on a full batch, with the residual.
        {"name": "rmsnorm_fwd_7B", "op": "rmsnorm", "dir": "fwd", "M": 8192, "d": 4096, "resid": True},
        # The same norm for a single token of a 70B-wide block.
        {"name": "rmsnorm_fwd_token", "op": "rmsnorm", "dir": "fwd", "M": 1, "d": 8192, "resid": True},
        # Its backward on a ragged batch, with a gradient arriving through the residual.
        {"name": "rmsnorm_bwd_7B_ragged", "op": "rmsnorm", "dir": "bwd", "M": 8000, "d": 4096, "resid": True},
        # Gate/up with SwiGLU on a full 7B batch, [a | b] kept in 8 bits for the backward.
        {"name": "swiglu_fwd_7B", "op": "swiglu", "dir": "fwd", "M": 8192, "K": 4096, "F": 11008, "save": True},
        # The same for a decoding step of the 1B block: nothing is kept.
        {"name": "swiglu_fwd_decode_1B", "op": "swiglu", "dir": "fwd", "M": 16, "K": 2048, "F": 8192,
         "save": False},
        # The SwiGLU backward from the 8-bit checkpoint, all operands of dgrad and wgrad, ragged tokens.
        {"name": "swiglu_bwd_7B_ragged", "op": "swiglu", "dir": "bwd", "M": 8190, "K": 4096, "F": 11008,
         "save": True},
        # An output gradient quantised both ways at once (for dgrad and for wgrad).
        {"name": "quant_grad_7B", "op": "quant", "dir": "rowscols", "M": 8191, "N": 4096, "type": "e5m2"},
        # The stacked gate/up weight of the 7B block after an optimiser step.
        {"name": "quant_weight_7B", "op": "quant", "dir": "blocks", "M": 22016, "N": 4096, "type": "e4m3"},
    ]


def draw(rng):
    def size(lo, hi, step=1):
        return step * max(1, round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step))

    op = rng.choice(("gemm", "gemm", "rmsnorm", "swiglu", "swiglu", "quant"))
    if op == "gemm":
        way = rng.choice(("fwd", "dgrad", "wgrad"))
        kind = rng.choice(("e4m3", "e5m2")) if way != "fwd" else "e4m3"
        if way == "wgrad":
            return {"op": op, "dir": way, "M": size(256, 8192, 16), "N": size(256, 8192, 16),
                    "K": size(1, 8192), "type": kind}
        return {"op": op, "dir": way, "M": size(1, 8192), "N": size(256, 8192, 16), "K": size(256, 11008, 16),
                "type": kind}
    if op == "rmsnorm":
        return {"op": op, "dir": rng.choice(("fwd", "bwd")), "M": size(1, 16384), "d": size(256, 8192, 16),
                "resid": rng.random() < 0.7}
    if op == "swiglu":
        way = rng.choice(("fwd", "bwd"))
        return {"op": op, "dir": way, "M": size(1, 8192), "K": size(256, 4096, 16), "F": size(256, 11008, 128),
                "save": way == "bwd" or rng.random() < 0.6}
    way = rng.choice(("rowscols", "rows", "blocks"))
    return {"op": op, "dir": way, "M": size(1, 16384), "N": size(256, 11008, 16),
            "type": rng.choice(("e4m3", "e5m2"))}


# ------------------------------------------------------------------ 8-bit blocks, plain

def _pad(x, rows, cols):
    """x [R, C] with zeros up to whole blocks of rows x cols (a zero never raises a block's amax)."""
    return torch.nn.functional.pad(x, (0, -x.shape[1] % cols, 0, -x.shape[0] % rows))


def _quant(x, rows, cols, kind):
    """Blocks of rows x cols of x (fp32): the 8-bit values [R, C] and the scales [blocks of R, blocks of C]."""
    dtype, fmax = TYPES[kind]
    R, C = x.shape
    p = _pad(x, rows, cols)
    t = p.view(p.shape[0] // rows, rows, p.shape[1] // cols, cols)
    amax = t.abs().amax(dim=(1, 3)).clamp_min(TINY)
    q = (t * (fmax / amax)[:, None, :, None]).clamp(-fmax, fmax)
    return q.view(p.shape)[:R, :C].contiguous().to(dtype), amax / fmax


def _rows(x, kind="e4m3"):
    q, s = _quant(x, 1, 128, kind)
    return q, s.t().contiguous()


def _cols(x, kind="e4m3"):
    return _quant(x, 128, 1, kind)


def _unrows(q, s, dtype=torch.float32):
    return q.to(dtype) * s.to(dtype).t().repeat_interleave(128, 1)[:, :q.shape[1]]


def _uncols(q, s, dtype=torch.float32):
    return q.to(dtype) * s.to(dtype).repeat_interleave(128, 0)[:q.shape[0]]


def _unblocks(q, s, dtype=torch.float32):
    s = s.to(dtype).repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :q.shape[1]]
    return q.to(dtype) * s


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    def activations(rows, cols):
        """Normal values with a few wide channels, as a residual stream has them."""
        wide = torch.rand(cols, device="cuda", generator=gen) < 1.0 / 256
        return normal(rows, cols) * (1.0 + 7.0 * wide)

    s = dict(case)
    op, way = case["op"], case["dir"]
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        if way == "wgrad":
            s["A"], s["SA"] = _cols(normal(K, M), case["type"])
            s["B"], s["SB"] = _cols(activations(K, N))
        else:
            s["A"], s["SA"] = _rows(activations(M, K), case["type"])
            w = normal(N, K) if way == "fwd" else normal(K, N)
            s["B"], s["SB"] = _quant(w * K ** -0.5, 128, 128, "e4m3")
    elif op == "rmsnorm":
        M, d = case["M"], case["d"]
        s["X"] = activations(M, d).bfloat16()
        s["R"] = normal(M, d).bfloat16() if case["resid"] else None
        s["g"] = (1.0 + 0.1 * normal(d)).bfloat16()
        if way == "bwd":
            s["dN"] = (normal(M, d) * 0.02).bfloat16()
            s["r"] = torch.rsqrt(s["X"].float().square().mean(1) + 1e-6)
    elif op == "swiglu":
        M, K, F = case["M"], case["K"], case["F"]
        if way == "fwd":
            s["A"], s["SA"] = _rows(activations(M, K))
            s["W"], s["SW"] = _quant(normal(2 * F, K) * K ** -0.5, 128, 128, "e4m3")
        else:
            s["AB"], s["SAB"] = _rows(normal(M, 2 * F) * 1.2)
            s["dY"] = (normal(M, F) * 0.02).bfloat16()
    else:
        x = normal(case["M"], case["N"])
        s["X"] = (x * (case["N"] ** -0.5 if way == "blocks" else 0.02)).bfloat16()
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    from gemm_epilogue_fusion_tmem_b200 import binding as coda

    op, way = s["op"], s["dir"]
    if op == "gemm":
        if way == "wgrad":
            return coda.gemm_fp8(s["A"], s["SA"], s["B"], s["SB"], s["M"], s["N"], s["K"], a_mn_major=True,
                                 b_mn_major=True, b_blocks=False, out_dtype=torch.float32)
        return coda.gemm_fp8(s["A"], s["SA"], s["B"], s["SB"], s["M"], s["N"], s["K"], b_mn_major=way == "dgrad")
    if op == "rmsnorm":
        if way == "fwd":
            return coda.rmsnorm_fp8_fwd(s["X"], s["g"], 1e-6, R=s["R"])
        return coda.rmsnorm_fp8_bwd(s["dN"], s["X"], s["r"], s["g"], dH_in=s["R"])
    if op == "swiglu":
        if way == "fwd":
            return coda.gemm_swiglu_fp8(s["A"], s["SA"], s["W"], s["SW"], save_ab=s["save"])
        return coda.swiglu_fp8_bwd(s["dY"], s["AB"], s["SAB"])
    if way == "blocks":
        return coda.quant_fp8_blocks(s["X"], fmt=TYPES[s["type"]][0])
    return coda.quant_fp8(s["X"], cols=way == "rowscols", fmt=TYPES[s["type"]][0])


def _plain(s):
    op, way = s["op"], s["dir"]
    if op == "gemm":
        if way == "fwd":
            return (_unrows(s["A"], s["SA"]) @ _unblocks(s["B"], s["SB"]).t()).bfloat16()
        if way == "dgrad":
            return (_unrows(s["A"], s["SA"]) @ _unblocks(s["B"], s["SB"])).bfloat16()
        return _uncols(s["A"], s["SA"]).t() @ _uncols(s["B"], s["SB"])
    if op == "rmsnorm":
        g = s["g"].float()
        if way == "fwd":
            o = {}
            h = s["X"]
            if s["R"] is not None:
                h = o["H"] = (h.float() + s["R"].float()).bfloat16()
            h = h.float()
            o["r"] = torch.rsqrt(h.square().mean(1) + 1e-6)
            o["Q"], o["S"] = _rows(h * o["r"][:, None] * g)
            return o
        dn, h, r = s["dN"].float(), s["X"].float(), s["r"][:, None]
        u = dn * g
        dh = r * u - h * r.pow(3) * (u * h).mean(1, keepdim=True)
        if s["R"] is not None:
            dh = dh + s["R"].float()
        return {"dH": dh.bfloat16(), "dg": (dn * h * r).sum(0, dtype=torch.float64).float()}
    if op == "swiglu":
        if way == "fwd":
            ab = _unrows(s["A"], s["SA"]) @ _unblocks(s["W"], s["SW"]).t()
            a, b = ab.chunk(2, 1)
            o = {}
            o["Y"], o["SY"] = _rows(a * torch.sigmoid(a) * b)
            if s["save"]:
                o["AB"], o["SAB"] = _rows(ab)
            return o
        a, b = _unrows(s["AB"], s["SAB"]).chunk(2, 1)
        dy = s["dY"].float()
        sg = torch.sigmoid(a)
        dab = torch.cat((dy * b * sg * (1.0 + a * (1.0 - sg)), dy * a * sg), 1)
        o = {}
        o["dA"], o["SdA"] = _rows(dab)
        o["dAc"], o["SdAc"] = _cols(dab)
        o["Yc"], o["SYc"] = _cols(a * sg * b)
        return o
    x, o = s["X"].float(), {}
    if way == "blocks":
        o["Q"], o["S"] = _quant(x, 128, 128, s["type"])
        return o
    o["Qr"], o["Sr"] = _rows(x, s["type"])
    if way == "rowscols":
        o["Qc"], o["Sc"] = _cols(x, s["type"])
    return o


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op, way = case["op"], case["dir"]
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        kb = _cdiv(K, 128)
        sb = kb * N if way == "wgrad" else kb * _cdiv(N, 128)
        out = (4 if way == "wgrad" else 2) * M * N
        return {"bytes": M * K + N * K + 4 * kb * M + 4 * sb + out, "flops": 2 * M * N * K}
    if op == "rmsnorm":
        M, d = case["M"], case["d"]
        if way == "fwd":
            return {"bytes": M * d * (2 + (4 if case["resid"] else 0) + 1) + 4 * M * (1 + _cdiv(d, 128)) + 2 * d,
                    "flops": 6 * M * d}
        return {"bytes": M * d * (6 + (2 if case["resid"] else 0)) + 4 * M + 6 * d, "flops": 10 * M * d}
    if op == "swiglu":
        M, K, F = case["M"], case["K"], case["F"]
        fb, kb, mb = F // 128, _cdiv(K, 128), _cdiv(M, 128)
        if way == "fwd":
            keep = 2 * M * F + 8 * fb * M if case["save"] else 0
            return {"bytes": M * K + 2 * F * K + 4 * kb * (M + 2 * fb) + M * F + 4 * fb * M + keep,
                    "flops": 4 * M * K * F}
        return {"bytes": 9 * M * F + 16 * fb * M + 12 * F * mb, "flops": 25 * M * F}
    M, N = case["M"], case["N"]
    if way == "blocks":
        return {"bytes": 3 * M * N + 4 * _cdiv(M, 128) * _cdiv(N, 128), "flops": 2 * M * N}
    both = way == "rowscols"
    return {"bytes": M * N * (4 if both else 3) + 4 * M * _cdiv(N, 128) + (4 * N * _cdiv(M, 128) if both else 0),
            "flops": (4 if both else 2) * M * N}


# ------------------------------------------------------------------ the definition in 64 bits

def _nearest(x, kind):
    """The nearest 8-bit number of each value of x (fp64, ties to the even one)."""
    bits, low = (3, -6) if kind == "e4m3" else (2, -14)
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp_min(low) - bits)
    return torch.round(x / step) * step


def _exact_blocks(x, rows, cols, kind):
    top = 448.0 if kind == "e4m3" else 57344.0
    R, C = x.shape
    big = torch.nn.functional.max_pool2d(x.abs()[None, None], (rows, cols), ceil_mode=True)[0, 0].clamp_min(TINY)
    each = big.repeat_interleave(rows, 0)[:R].repeat_interleave(cols, 1)[:, :C]
    return _nearest(x * (top / each), kind), big / top


def _exact_rows(x, kind="e4m3"):
    q, s = _exact_blocks(x, 1, 128, kind)
    return q, s.t()


def _spread(s, rows, cols, R, C):
    return s.double().repeat_interleave(rows, 0)[:R].repeat_interleave(cols, 1)[:, :C]


def exact(case, seed):
    s = prepare(case, seed)
    op, way = case["op"], case["dir"]
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        A, B = s["A"].double(), s["B"].double()
        if way == "wgrad":
            return (A * _spread(s["SA"], 128, 1, K, M)).t().matmul(B * _spread(s["SB"], 128, 1, K, N))
        A = A * _spread(s["SA"].t(), 1, 128, M, K)
        if way == "fwd":
            return A.matmul((B * _spread(s["SB"], 128, 128, N, K)).t())
        return A.matmul(B * _spread(s["SB"], 128, 128, K, N))
    if op == "rmsnorm":
        g = s["g"].double()
        if way == "fwd":
            o, h = {}, s["X"].double()
            if s["R"] is not None:
                h = o["H"] = h + s["R"].double()
                h = h.bfloat16().double()  # the norm is of the stored sum
            o["r"] = (h.pow(2).sum(1) / case["d"] + 1e-6).pow(-0.5)
            o["Q"], o["S"] = _exact_rows(h * g * o["r"].unsqueeze(1))
            return o
        dn, h, r = s["dN"].double(), s["X"].double(), s["r"].double().unsqueeze(1)
        n = h * r
        u = dn * g
        dh = (u - n * (u * n).sum(1, keepdim=True) / case["d"]) * r
        if s["R"] is not None:
            dh = dh + s["R"].double()
        return {"dH": dh, "dg": (dn * n).sum(0)}
    if op == "swiglu":
        M, K, F = case["M"], case["K"], case["F"]
        if way == "fwd":
            A = s["A"].double() * _spread(s["SA"].t(), 1, 128, M, K)
            ab = A.matmul((s["W"].double() * _spread(s["SW"], 128, 128, 2 * F, K)).t())
            a, b = ab[:, :F], ab[:, F:]
            o = {}
            o["Y"], o["SY"] = _exact_rows(a * b / (1.0 + torch.exp(-a)))
            if case["save"]:
                o["AB"], o["SAB"] = _exact_rows(ab)
            return o
        ab = s["AB"].double() * _spread(s["SAB"].t(), 1, 128, M, 2 * F)
        a, b, dy = ab[:, :F], ab[:, F:], s["dY"].double()
        p = 1.0 / (1.0 + torch.exp(-a))
        dab = torch.cat((dy * b * (p + a * p * (1.0 - p)), dy * a * p), 1)
        o = {}
        o["dA"], o["SdA"] = _exact_rows(dab)
        o["dAc"], o["SdAc"] = _exact_blocks(dab, 128, 1, "e4m3")
        o["Yc"], o["SYc"] = _exact_blocks(a * b * p, 128, 1, "e4m3")
        return o
    x, o = s["X"].double(), {}
    if way == "blocks":
        o["Q"], o["S"] = _exact_blocks(x, 128, 128, case["type"])
        return o
    o["Qr"], o["Sr"] = _exact_rows(x, case["type"])
    if way == "rowscols":
        o["Qc"], o["Sc"] = _exact_blocks(x, 128, 1, case["type"])
    return o
