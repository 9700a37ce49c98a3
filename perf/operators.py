"""The operators around a quantised stack: token rows in, next tokens out.

A pass is one call of one operator, with the inputs a decoding program holds:

  norm     r = x + residual, RMSNorm, 8-bit codes with scales   (lib.add_norm_quant)
  gemm     e4m3 product with a scale per block of 128           (lib.fp8_gemm)
  beam     the n best of beams x vocabulary                     (lib.beam_select)
  reorder  the beams' carried states follow their parents       (lib.reorder_rows)
  embed    scaled table rows of the chosen tokens               (lib.embed_rows)

Where `own` is false, run() computes the plain form with elementary torch
operations; where it is true it calls the framework.  exact() is the
definition in 64 bits, written apart from the plain form.
"""
import math

import torch

own = False

CODE_MAX = {"e4m3": 448.0, "int8": 127.0}
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn,
          "int8": torch.int8, "int16": torch.int16, "int32": torch.int32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode batch of 64 sequences in front of the output head (2.7B width)
        dict(name="norm decode 64x2560", op="norm", M=64, K=2560, x="fp32", out="e4m3", residual=True),
        # the residual stream of a 2 x 4096 prompt at the same width
        dict(name="norm prompt 8192x2560", op="norm", M=8192, K=2560, x="fp32", out="e4m3",
             residual=True),
        # int8 codes for the W8A8 linears, bf16 rows, an odd token count (130M width)
        dict(name="norm int8 2049x768", op="norm", M=2049, K=768, x="bf16", out="int8", residual=True),
        # the output head for 4 beams of one sequence, an odd vocabulary
        dict(name="head 4x32001x768", op="gemm", M=4, N=32001, K=768, y="fp32"),
        # the output head for a batch of 64 rows: the weights' bytes bound it
        dict(name="head 64x50000x2560", op="gemm", M=64, N=50000, K=2560, y="fp32"),
        # a projection of a long prompt (the 2.7B in_proj's sizes): the tensor cores bound it
        dict(name="projection 8192x10576x2560", op="gemm", M=8192, N=10576, K=2560, y="bf16"),
        # one sequence, four beams: latency
        dict(name="beam 1x4x32001", op="beam", B=1, beams=4, n_out=4, V=32001, logits="fp32",
             finished=False),
        # a batch of 64 with 8 beams, some of them finished, forbidden tokens at -inf
        dict(name="beam 64x8x100003", op="beam", B=64, beams=8, n_out=8, V=100003, logits="bf16",
             finished=True),
        # the states of a 24-layer 130M stack, one sequence of 4 beams, 16-bit state
        dict(name="reorder 24 layers 1x4", op="reorder", layers=24, B=1, beams=4, d_inner=1536,
             state="int16", expand=False),
        # the states of a 64-layer 2.7B stack, 4 sequences of 8 beams
        dict(name="reorder 64 layers 4x8", op="reorder", layers=64, B=4, beams=8, d_inner=5120,
             state="int32", expand=False),
        # the chosen tokens of 64 rows from an 8-bit table that is the output head's weight too
        dict(name="embed decode 64x2560", op="embed", M=64, V=50000, K=2560, table="e4m3"),
        # a 2 x 4096 prompt from a bf16 table, padded with id -1
        dict(name="embed prompt 8192x2560", op="embed", M=8192, V=50000, K=2560, table="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "gemm", "beam", "reorder", "embed"])
    if op == "norm":
        return dict(op=op, M=_log(rng, 1, 8192), K=16 * _log(rng, 4, 160),
                    x=rng.choice(["fp32", "bf16"]), out=rng.choice(["e4m3", "int8"]),
                    residual=rng.random() < 0.7)
    if op == "gemm":
        M, K = _log(rng, 1, 8192), 16 * _log(rng, 16, 320)
        N = _log(rng, 1, min(50000, 8192 * 10576 * 2560 // (M * K)))
        return dict(op=op, M=M, N=N, K=K, y=rng.choice(["fp32", "bf16"]))
    if op == "beam":
        beams = rng.randint(1, 16)
        B = _log(rng, 1, max(1, 512 // beams))
        V = _log(rng, 40, 100003)
        return dict(op=op, B=B, beams=beams, n_out=rng.choice([beams, rng.randint(1, 16)]), V=V,
                    logits=rng.choice(["fp32", "bf16"]) if B * beams <= 256 else "bf16",
                    finished=rng.random() < 0.5)
    if op == "reorder":
        beams = rng.randint(2, 16)
        return dict(op=op, layers=rng.randint(1, 32), B=_log(rng, 1, max(1, 32 // beams)), beams=beams,
                    d_inner=256 * rng.randint(1, 20), state=rng.choice(["int16", "int32"]),
                    expand=rng.random() < 0.3)
    return dict(op=op, M=_log(rng, 1, 8192), V=_log(rng, 2, 50000), K=16 * _log(rng, 4, 160),
                table=rng.choice(["fp32", "bf16", "e4m3"]))


def _blocks(n):
    return (n + 127) // 128


def _state_bytes(c):
    """(bytes of one row's conv state, bytes of one row's scan state)"""
    return 3 * (c["d_inner"] + 256), c["d_inner"] * 128 * (2 if c["state"] == "int16" else 4)


def work(case):
    c, size = case, {"fp32": 4, "bf16": 2, "e4m3": 1, "int8": 1}
    if c["op"] == "norm":
        n = c["M"] * c["K"]
        scales = 4 * c["M"] * (_blocks(c["K"]) if c["out"] == "e4m3" else 1)
        return {"bytes": n * (size[c["x"]] + 1 + (8 if c["residual"] else 0)) + scales + 4 * c["K"],
                "flops": 6 * n}
    if c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": M * K + N * K + 4 * _blocks(K) * (M + _blocks(N)) + M * N * size[c["y"]],
                "flops": 2 * M * N * K}
    if c["op"] == "beam":
        n = c["B"] * c["beams"] * c["V"]
        return {"bytes": n * size[c["logits"]] + c["B"] * (5 * c["beams"] + 13 * c["n_out"]),
                "flops": 4 * n}
    if c["op"] == "reorder":
        row, G = c["layers"] * sum(_state_bytes(c)), c["beams"]
        if c["expand"]:  # one source row for every G
            return {"bytes": c["B"] * row * (1 + G), "flops": 0}
        # parents are uniform: the rows whose parent is another beam are
        # written, the beams that are another's parent are read
        written, read = 1 - 1 / G, 1 - (1 - 1 / G) ** (G - 1)
        return {"bytes": int(c["B"] * G * row * (written + read)), "flops": 0}
    n = c["M"] * c["K"]
    scales = 4 * c["M"] * _blocks(c["K"]) if c["table"] == "e4m3" else 0
    return {"bytes": n * (size[c["table"]] + 4) + scales + 4 * c["M"], "flops": 2 * n}


# ------------------------------------------------------------------ inputs
def _block_codes(w, rows):
    """e4m3 codes of w [R, K] and its scales: one per `rows` rows and 128 columns."""
    R, K = w.shape
    nr, nk = (R + rows - 1) // rows, _blocks(K)
    p = torch.zeros(nr * rows, nk * 128, device=w.device)
    p[:R, :K] = w
    p = p.view(nr, rows, nk, 128)
    s = p.abs().amax(dim=(1, 3)).clamp_min(1e-30) / 448.0
    q = (p / s[:, None, :, None]).to(torch.float8_e4m3fn)
    return q.view(nr * rows, nk * 128)[:R, :K].contiguous(), s.contiguous()


def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed * 7919 + 13)

    def normal(*shape):
        return torch.randn(*shape, device=dev, generator=g)

    def empty(*shape, dtype=torch.float32):
        return torch.empty(*shape, device=dev, dtype=dtype)

    if c["op"] == "norm":
        M, K = c["M"], c["K"]
        x = normal(M, K)
        x[:, torch.randperm(K, device=dev, generator=g)[:max(1, K // 96)]] *= 50.0  # outlier channels
        c.update(x_=x.to(DTYPES[c["x"]]), w_=1.0 + 0.1 * normal(K),
                 r_=3.0 * normal(M, K) if c["residual"] else None,
                 sum_=empty(M, K) if c["residual"] else None,
                 q_=empty(M, K, dtype=DTYPES[c["out"]]),
                 s_=empty(M, _blocks(K)) if c["out"] == "e4m3" else empty(M))
    elif c["op"] == "gemm":
        a, sa = _block_codes(normal(c["M"], c["K"]), 1)
        w, sw = _block_codes(0.02 * normal(c["N"], c["K"]), 128)
        c.update(a_=a, sa_=sa, w_=w, sw_=sw, y_=empty(c["M"], c["N"], dtype=DTYPES[c["y"]]))
    elif c["op"] == "beam":
        B, k, V, n = c["B"], c["beams"], c["V"], c["n_out"]
        logits = 2.5 * normal(B, k, V)
        logits[:, :, torch.randint(0, V, (max(1, V // 50),), device=dev, generator=g)] = -math.inf
        scores = -torch.rand(B, k, device=dev, generator=g).cumsum(1) - 5.0
        fin = torch.rand(B, k, device=dev, generator=g) < 0.2 if c["finished"] else None
        i32 = torch.int32
        c.update(logits_=logits.to(DTYPES[c["logits"]]), scores_=scores,
                 fin_=fin.to(torch.uint8) if fin is not None else None,
                 eos=int(V // 2) if fin is not None else -1, out_=empty(B, n),
                 parent_=empty(B, n, dtype=i32), token_=empty(B, n, dtype=i32),
                 nfin_=empty(B, n, dtype=torch.uint8) if fin is not None else None)
        if own:
            from quantized_state_space_mamba2_b200 import lib
            c["ws_"] = empty(lib.beam_workspace_bytes(B, k, V, n), dtype=torch.uint8)
    elif c["op"] == "reorder":
        L, B, G, di = c["layers"], c["B"], c["beams"], c["d_inner"]
        rows, lim = B * (1 if c["expand"] else G), 20000

        def ints(dtype, *shape):
            return torch.randint(-lim if dtype != torch.int8 else -127,
                                 lim if dtype != torch.int8 else 128, shape, device=dev,
                                 generator=g, dtype=dtype)

        c.update(conv_=ints(torch.int8, L, rows, 3, di + 256),
                 ssm_=ints(DTYPES[c["state"]], L, rows, di // 64, 64, 128))
        c["conv_out_"] = empty(L, B * G, 3, di + 256, dtype=torch.int8) if c["expand"] else c["conv_"]
        c["ssm_out_"] = (empty(L, B * G, di // 64, 64, 128, dtype=DTYPES[c["state"]])
                         if c["expand"] else c["ssm_"])
        c["parent_"] = torch.randint(0, 1 if c["expand"] else G, (B, G), device=dev, generator=g,
                                     dtype=torch.int32)
        if own:  # the handle that a decoding program makes once for its state buffers
            from quantized_state_space_mamba2_b200 import lib
            c["rows_"] = lib.RowSet([t for l in range(L) for t in (c["conv_out_"][l], c["ssm_out_"][l])],
                                    [t for l in range(L) for t in (c["conv_"][l], c["ssm_"][l])])
    else:
        ids = torch.randint(0, c["V"], (c["M"],), device=dev, generator=g, dtype=torch.int32)
        ids[torch.rand(c["M"], device=dev, generator=g) < 0.05] = -1  # padding
        t, ts = 0.02 * normal(c["V"], c["K"]), None
        if c["table"] == "e4m3":
            t, ts = _block_codes(t, 128)
        c.update(ids_=ids, t_=t.to(DTYPES[c["table"]]), ts_=ts, scale=math.sqrt(c["K"]),
                 x_=empty(c["M"], c["K"]))
    return c


# ------------------------------------------------------------------ one pass
def run(state):
    return (_own if own else _plain)(state)


def _own(c):
    from quantized_state_space_mamba2_b200 import lib
    if c["op"] == "norm":
        lib.add_norm_quant(c["x_"], c["w_"], c["q_"], c["s_"], residual=c["r_"], sum_out=c["sum_"])
        return _norm_out(c["q_"], c["s_"], c["sum_"])
    if c["op"] == "gemm":
        lib.fp8_gemm(c["a_"], c["sa_"], c["w_"], c["sw_"], c["y_"])
        return c["y_"]
    if c["op"] == "beam":
        lib.beam_select(c["logits_"], c["scores_"], c["out_"], c["parent_"], c["token_"], c["ws_"],
                        finished=c["fin_"], out_finished=c["nfin_"], eos=c["eos"])
        return {"score": c["out_"], "parent": c["parent_"], "token": c["token_"], "fin": c["nfin_"]}
    if c["op"] == "reorder":
        lib.reorder_rows(c["rows_"], c["parent_"], src_beams=1 if c["expand"] else None)
        return {"conv": c["conv_out_"], "ssm": c["ssm_out_"]}
    lib.embed_rows(c["ids_"], c["t_"], c["x_"], table_s=c["ts_"], scale=c["scale"])
    return c["x_"]


def _norm_out(q, s, r):
    # codes are returned as the (unscaled) values they stand for: e4m3 as they
    # are, int8 as whole numbers
    return {"codes": q, "scales": s} if r is None else {"codes": q, "scales": s, "sum": r}


def _plain(c):
    if c["op"] == "norm":
        # in 64 bits: a code is the nearest one, and near a border between two
        # codes 32 bits do not tell which that is
        r = c["x_"].float()
        if c["r_"] is not None:
            r = r + c["r_"]
        d = r.double()
        y = d * torch.rsqrt(d.square().mean(1, keepdim=True) + 1e-5) * c["w_"].double()
        M, K = y.shape
        if c["out"] == "int8":
            s = (y.abs().amax(1, keepdim=True) / 127.0).float()
            q = torch.round(y / s.double()).clamp(-127, 127).to(torch.int8)
            return _norm_out(q, s[:, 0], None if c["r_"] is None else r)
        y = torch.nn.functional.pad(y, (0, _blocks(K) * 128 - K)).view(M, -1, 128)
        s = (y.abs().amax(2, keepdim=True) / 448.0).float()
        v = y / s.double()
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3.0)
        q = (torch.round(v / step) * step).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        return _norm_out(q.view(M, -1)[:, :K], s[:, :, 0], None if c["r_"] is None else r)
    if c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        a = c["a_"].float() * c["sa_"].repeat_interleave(128, 1)[:, :K]
        w = c["w_"].float() * c["sw_"].repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
        return (a @ w.t()).to(DTYPES[c["y"]])
    if c["op"] == "beam":
        # in 64 bits: the order of two candidates is a border
        B, k, V, n = c["B"], c["beams"], c["V"], c["n_out"]
        l = c["logits_"].double()
        top = l.amax(2, keepdim=True)
        lse = top + torch.exp(l - top).sum(2, keepdim=True).log()
        cand = l - lse + c["scores_"].double()[:, :, None]
        fin = torch.zeros(B, k, dtype=torch.bool, device=l.device)
        if c["fin_"] is not None:  # a finished beam goes on as it is, at eos
            fin = c["fin_"].bool()
            stay = torch.arange(V, device=l.device) == c["eos"]
            frozen = torch.where(stay, c["scores_"].double()[:, :, None], -math.inf)
            cand = torch.where(fin[:, :, None], frozen, cand)
        v, i = torch.sort(cand.view(B, k * V), dim=1, descending=True, stable=True)
        v, i = v[:, :n], i[:, :n]
        if v.shape[1] < n:
            v = torch.nn.functional.pad(v, (0, n - v.shape[1]), value=-math.inf)
            i = torch.nn.functional.pad(i, (0, n - i.shape[1]))
        none = v == -math.inf
        slot = (torch.arange(n, device=l.device) % k).expand(B, n)
        parent, token = torch.where(none, slot, i // V), torch.where(none, -1, i % V)
        ended = None
        if c["fin_"] is not None:
            ended = (~none & (torch.gather(fin, 1, parent) | (token == c["eos"]))).to(torch.uint8)
        return {"score": v.float(), "parent": parent.int(), "token": token.int(), "fin": ended}
    if c["op"] == "reorder":
        B, G, L = c["B"], c["beams"], c["layers"]
        src = (torch.arange(B, device="cuda")[:, None] * (1 if c["expand"] else G)
               + c["parent_"]).view(-1)
        c["conv_out_"].copy_(c["conv_"].index_select(1, src))
        c["ssm_out_"].copy_(c["ssm_"].index_select(1, src))
        return {"conv": c["conv_out_"], "ssm": c["ssm_out_"]}
    ids, K = c["ids_"].long(), c["K"]
    at = ids.clamp_min(0)
    x = c["t_"][at].float()
    if c["ts_"] is not None:
        x = x * c["ts_"][at // 128].repeat_interleave(128, 1)[:, :K]
    return torch.where(ids[:, None] >= 0, x * c["scale"], 0.0)


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    c = prepare(case, seed)
    f64 = torch.float64
    if c["op"] == "norm":
        # r is an fp32 output; the codes are those nearest to y / s for the
        # fp32 scales s that go with them
        x = c["x_"].to(f64)
        r = (x + c["r_"].to(f64)).float() if c["r_"] is not None else x.float()
        M, K = r.shape
        y = r.to(f64) / (r.to(f64).pow(2).sum(1, keepdim=True) / K + 1e-5).sqrt() * c["w_"].to(f64)
        width = 128 if c["out"] == "e4m3" else K
        n = -(-K // width)
        codes, scales = torch.empty(M, K, dtype=f64, device=y.device), []
        for b in range(n):
            part = y[:, b * width:(b + 1) * width]
            s = (part.abs().max(1).values / CODE_MAX[c["out"]]).float().to(f64)
            v = part / s[:, None]
            if c["out"] == "e4m3":
                m, e = torch.frexp(v)  # |v| = m 2^e, m in [0.5, 1): 3 bits after the first
                unit = torch.ldexp(torch.ones_like(v), torch.maximum(e - 1, torch.full_like(e, -6)) - 3)
                v = torch.round(v / unit) * unit
            else:
                v = torch.round(v)
            codes[:, b * width:(b + 1) * width] = v
            scales.append(s)
        scales = torch.stack(scales, 1) if c["out"] == "e4m3" else scales[0]
        return _norm_out(codes, scales, None if c["r_"] is None else r.to(f64))
    if c["op"] == "gemm":
        y = torch.zeros(c["M"], c["N"], dtype=f64, device=c["a_"].device)
        scale_w = c["sw_"].to(f64)[torch.arange(c["N"], device=y.device) // 128]
        for b in range(_blocks(c["K"])):
            at = slice(128 * b, 128 * b + 128)
            a = c["a_"][:, at].to(f64) * c["sa_"][:, b:b + 1].to(f64)
            y += a @ (c["w_"][:, at].to(f64) * scale_w[:, b:b + 1]).t()
        return y
    if c["op"] == "beam":
        B, k, V, n = c["B"], c["beams"], c["V"], c["n_out"]
        logp = torch.log_softmax(c["logits_"].to(f64), dim=2) + c["scores_"].to(f64)[:, :, None]
        if c["fin_"] is not None:
            done = c["fin_"] != 0
            logp[done] = -math.inf
            logp[:, :, c["eos"]] = torch.where(done, c["scores_"].to(f64), logp[:, :, c["eos"]])
        best = logp.reshape(B, k * V).topk(min(n, k * V), dim=1).values
        score = torch.full((B, n), -math.inf, dtype=f64, device=best.device)
        score[:, :best.shape[1]] = best
        return {"score": score, "parent": None, "token": None, "fin": None}
    if c["op"] == "reorder":
        return None  # values are moved, none is computed
    ids, K = c["ids_"].long(), c["K"]
    x = torch.zeros(c["M"], K, dtype=f64, device=ids.device)
    live = (ids >= 0).nonzero()[:, 0]
    rows = c["t_"].to(torch.float32)[ids[live]].to(f64)
    if c["ts_"] is not None:
        rows = rows * c["ts_"].to(f64)[ids[live] // 128][:, torch.arange(K, device=ids.device) // 128]
    x[live] = rows * c["scale"]
    return x
