"""Measured cases of the softmax-attention operators: prompt attention (forward and gradients), the
write into the 8-bit paged cache and the decode attention that reads it.

A pass is run(prepare(case, seed)).  With own = False it computes the operators from elementary
torch operations in fp32; with own = True it calls the library.  exact() gives the same outputs
from the definitions in fp64."""
import math

import torch

own = False

DEV = "cuda:0"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
E4M3_MAX = 448.0
EXP_MIN, EXP_MAX = -100, 120  # exponent range of a cache scale


def listed():
    return [
        # a few short prompts admitted between decode steps: launch latency counts
        dict(name="prefill_small_fp32", op="prefill", lens_q="1,33,7,95", lens_k="1,33,7,95",
             H=8, Hk=2, dk=64, dv=64, dtype="fp32"),
        # an fp32 evaluation of two middling prompts, one kv head per query head
        dict(name="prefill_mid_fp32", op="prefill", lens_q="1501,700", lens_k="1501,700",
             H=16, Hk=16, dk=64, dv=64, dtype="fp32"),
        # a serving batch: whole prompts packed with chunks that continue longer contexts
        dict(name="prefill_mixed", op="prefill", lens_q="1000,2049,512,64,1,0,777",
             lens_k="1000,2049,9000,4160,513,0,777", H=32, Hk=8, dk=128, dv=128, dtype="bf16"),
        # the benchmark's prompt of 8192 tokens, 32 heads
        dict(name="prefill_8192", op="prefill", lens_q="8192", lens_k="8192", H=32, Hk=8, dk=128,
             dv=128, dtype="bf16"),
        # gradients of a few short sequences in fp32 (a gradient check, a small fine-tuning batch)
        dict(name="backward_small_fp32", op="backward", lens_q="1,40,129", lens_k="1,40,129",
             H=4, Hk=2, dk=64, dv=64, dtype="fp32"),
        # a packed training batch of ragged documents
        dict(name="backward_ragged", op="backward", lens_q="700,1333,65,2000", lens_k="700,1333,65,2000",
             H=16, Hk=4, dk=128, dv=128, dtype="bf16"),
        # a training sequence of 8192 tokens, 32 heads
        dict(name="backward_8192", op="backward", lens_q="8192", lens_k="8192", H=32, Hk=8, dk=128,
             dv=128, dtype="bf16"),
        # the cache write of a decode step of 64 sequences
        dict(name="append_decode", op="append", lens="1*64", start=4000, block=64, Hk=8, dk=128,
             dv=128, dtype="bf16"),
        # the cache write of the long varlen prompts
        dict(name="append_prompt", op="append", lens="100000,16384,8192,3500", start=0, block=64,
             Hk=8, dk=128, dv=128, dtype="bf16"),
        # one short conversation, fp32 queries: launch latency counts
        dict(name="decode_small_fp32", op="decode", lens="700", T=1, block=16, H=8, Hk=2, dk=64,
             dv=64, dtype="fp32"),
        # the decode batch of 64 sequences of mixed contexts, two of them padding
        dict(name="decode_batch", op="decode", lens="16000:62,0,0", T=1, block=64, H=32, Hk=8, dk=128,
             dv=128, dtype="bf16"),
        # speculative verification of 4 tokens on a few very long contexts
        dict(name="decode_verify_long", op="decode", lens="100000,131072,65537,8192", T=4, block=128, H=32,
             Hk=8, dk=128, dv=128, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "backward", "append", "decode"])
    dk, dv = rng.choice([(64, 64), (128, 128), (128, 128), (64, 128), (128, 64)])
    Hk = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 8])
    H = Hk * G
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    case = dict(op=op, Hk=Hk, dk=dk, dv=dv, dtype=dtype)
    if op in ("prefill", "backward"):
        top = 8192 if dtype == "bf16" else 2048
        # pairs of all sequences times heads stay below the largest listed case's
        room = (8192 * 8192 / 2 * 32 if dtype == "bf16" else 2048 * 2048 / 2 * 16) / H
        lq, lk = [], []
        for _ in range(rng.randint(1, 6)):
            a = _log_int(rng, 1, top)
            b = a + (_log_int(rng, 1, 8192) if rng.random() < 0.3 else 0)
            if a * (b - a / 2) <= room:
                room -= a * (b - a / 2)
                lq.append(a)
                lk.append(b)
        if not lq:
            lq, lk = [333], [333]
        case.update(H=H, lens_q=",".join(map(str, lq)), lens_k=",".join(map(str, lk)))
    elif op == "append":
        if rng.random() < 0.5:
            lens = "%d*%d" % (rng.randint(1, 8), _log_int(rng, 1, 128))
        else:
            lens = ",".join(str(_log_int(rng, 1, 20000)) for _ in range(rng.randint(1, 5)))
        case.update(lens=lens, start=rng.choice([0, 1, _log_int(rng, 1, 5000)]),
                    block=rng.choice([16, 32, 64, 128]))
    else:
        n = _log_int(rng, 1, 64)
        top = max(2, min(131072, 1000000 // n))
        if rng.random() < 0.5:
            lens = "%d:%d" % (_log_int(rng, 1, top), n)
        else:
            lens = ",".join(str(_log_int(rng, 1, top)) for _ in range(min(n, 12)))
        case.update(H=H, lens=lens, T=rng.choice([1, 1, 2, 3, 4, 8]), block=rng.choice([16, 32, 64, 128]))
    return case


def _lens(text):
    """"a,b" lengths; "a*n" n times a; "a:n" n lengths drawn from 1..a."""
    out = []
    for part in text.split(","):
        if "*" in part:
            a, n = part.split("*")
            out += [int(a)] * int(n)
        elif ":" in part:
            a, n = (int(x) for x in part.split(":"))
            # fixed by the case, so that its work is
            out += [1 + (i * 7919 + 4001) * 104729 % a for i in range(n)]
        else:
            out.append(int(part))
    return out


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _blocks(case, lens):
    """Per sequence the blocks its tokens take, and the pool's size (some blocks stay unused)."""
    per = [-(-n // case["block"]) for n in lens]
    return per, sum(per) + 3


def _pairs(lens_q, lens_k):
    return sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(lens_q, lens_k))


def work(case):
    dk, dv, Hk = case["dk"], case["dv"], case["Hk"]
    b = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("prefill", "backward"):
        lq, lk = _lens(case["lens_q"]), _lens(case["lens_k"])
        H, tq, tk = case["H"], sum(lq), sum(lk)
        pairs = _pairs(lq, lk) * H
        if case["op"] == "prefill":
            return {"bytes": b * (tq * H * (dk + dv) + tk * Hk * (dk + dv)) + 4 * tq * H,
                    "flops": 2 * pairs * (dk + dv)}
        return {"bytes": b * (tq * H * (2 * dk + 2 * dv) + 2 * tk * Hk * (dk + dv)) + 4 * tq * H,
                "flops": 2 * pairs * (3 * dk + 2 * dv)}
    lens = _lens(case["lens"])
    if case["op"] == "append":
        n = sum(lens) * Hk * (dk + dv)
        per, _ = _blocks(case, lens)
        return {"bytes": n * (b + 1) + 8 * Hk * sum(per), "flops": 2 * n}
    T, H = case["T"], case["H"]
    per, _ = _blocks(case, lens)
    pairs = sum(max(0, n - T + t + 1) for n in lens for t in range(T)) * H
    return {"bytes": sum(lens) * Hk * (dk + dv) + 8 * Hk * sum(per) + 4 * sum(per)
            + b * len(lens) * T * H * (dk + dv), "flops": 2 * pairs * (dk + dv)}


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    dk, dv, Hk = case["dk"], case["dv"], case["Hk"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV).to(dt)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    s = dict(case=case, scale=dk ** -0.5)
    if case["op"] in ("prefill", "backward"):
        lq, lk, H = _lens(case["lens_q"]), _lens(case["lens_k"]), case["H"]
        s.update(lens_q=lq, lens_k=lk, q=normal(sum(lq), H, dk), k=normal(sum(lk), Hk, dk),
                 v=normal(sum(lk), Hk, dv), cu_q=ints(_cu(lq)), cu_k=ints(_cu(lk)))
        s["lse"] = torch.empty(sum(lq), H, dtype=torch.float32, device=DEV)
        if case["op"] == "backward":
            s["do"] = normal(sum(lq), H, dv)
            # the forward's outputs, which a training step has kept
            s["o"], s["lse"] = _prefill(s)
        return s
    lens = _lens(case["lens"])
    N, block = len(lens), case["block"]
    start = case["start"] if case["op"] == "append" else 0
    per, pool = _blocks(case, [n + start for n in lens])
    order = torch.randperm(pool, generator=g, device=DEV)[:sum(per)].tolist()
    table = torch.full((N, max(max(per), 1)), -1, dtype=torch.int32)
    at = 0
    for n, c in enumerate(per):
        table[n, :c] = torch.tensor(order[at:at + c], dtype=torch.int32)
        at += c
    s.update(lens=lens, table=table.to(DEV))
    # a cache in use: rows of N(0, 1) quantised by blocks, as earlier appends left them
    s["k_scale"] = torch.full((pool, Hk), 2.0 ** -6, device=DEV)
    s["v_scale"] = torch.full((pool, Hk), 2.0 ** -6, device=DEV)
    for name, shape in (("k_cache", (block, dk)), ("v_cache", (dv, block))):
        x = torch.randn(pool, Hk, *shape, generator=g, device=DEV).clamp_(-7, 7)
        s[name] = (x * 2.0 ** 6).to(torch.float8_e4m3fn)
    if case["op"] == "append":
        s.update(k=normal(sum(lens), Hk, dk), v=normal(sum(lens), Hk, dv), cu_q=ints(_cu(lens)),
                 start=[start] * N, start_len=ints([start] * N))
        if start % block:
            # half of the sequences meet values above those their last block was scaled for
            for n in range(0, N, 2):
                if lens[n]:
                    s["k"][sum(lens[:n])] *= 4
    else:
        s.update(q=normal(N, case["T"], case["H"], dk), context_len=ints(lens))
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        import kda_gated_delta_rule_amd as kda

        if op == "prefill":
            o = kda.attn_prefill(state["q"], state["k"], state["v"], state["cu_q"],
                                 cu_seqlens_k=state["cu_k"], lse=state["lse"], scale=state["scale"])
            return {"o": o, "lse": state["lse"]}
        if op == "backward":
            dq, dk, dv = kda.attn_backward(state["q"], state["k"], state["v"], state["o"],
                                           state["lse"], state["do"], state["cu_q"],
                                           cu_seqlens_k=state["cu_k"], scale=state["scale"])
            return {"dq": dq, "dk": dk, "dv": dv}
        if op == "append":
            kda.attn_cache_append(state["k"], state["v"], state["cu_q"], state["start_len"],
                                  state["k_cache"], state["v_cache"], state["k_scale"],
                                  state["v_scale"], state["table"], clear=True)
            return _cache(state)
        return {"o": kda.attn_decode(state["q"], state["k_cache"], state["v_cache"],
                                     state["k_scale"], state["v_scale"], state["table"],
                                     state["context_len"], scale=state["scale"])}
    if op == "prefill":
        o, lse = _prefill(state)
        return {"o": o, "lse": lse}
    if op == "backward":
        return _backward(state)
    if op == "append":
        _append(state)
        return _cache(state)
    return {"o": _decode(state)}


def _cache(state):
    # the e4m3 numbers and the power-of-two scales that they are multiples of
    return {n: state[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}


# ---------------------------------------------------------------------------
# plain forms, fp32
# ---------------------------------------------------------------------------
def _scores(q, k, scale, Lq, Lk):
    """q [G, Lq, dk], k [Lk, dk] -> scores [G, Lq, Lk], -inf where query i may not see key j."""
    s = torch.matmul(q, k.t()) * scale
    i = torch.arange(Lq, device=q.device)[:, None]
    j = torch.arange(Lk, device=q.device)[None, :]
    return s.masked_fill_(j > i + (Lk - Lq), float("-inf"))


def _softmax(s):
    """(p, lse) along the last axis; a row of -inf only gives p = 0, lse = -inf."""
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == float("-inf"), torch.zeros_like(m), m))
    z = p.sum(-1, keepdim=True)
    lse = (m + torch.log(z)).squeeze(-1)
    return p / torch.where(z == 0, torch.ones_like(z), z), lse


def _heads(state):
    """Per sequence with queries and keys and per kv head: its token and head ranges."""
    case = state["case"]
    G = case["H"] // case["Hk"]
    a = b = 0
    for Lq, Lk in zip(state["lens_q"], state["lens_k"]):
        if Lq and Lk:
            for h in range(case["Hk"]):
                yield slice(a, a + Lq), slice(b, b + Lk), slice(h * G, h * G + G), h, Lq, Lk
        a, b = a + Lq, b + Lk


def _prefill(state):
    q, k, v = (state[n] for n in ("q", "k", "v"))
    o = torch.zeros(q.shape[0], q.shape[1], v.shape[2], dtype=q.dtype, device=q.device)
    lse = torch.full(q.shape[:2], float("-inf"), dtype=torch.float32, device=q.device)
    for tq, tk, hq, h, Lq, Lk in _heads(state):
        s = _scores(q[tq, hq].float().transpose(0, 1).contiguous(), k[tk, h].float(), state["scale"],
                    Lq, Lk)
        p, z = _softmax(s)
        o[tq, hq] = torch.matmul(p, v[tk, h].float()).transpose(0, 1).to(o.dtype)
        lse[tq, hq] = z.t()
    return o, lse


def _backward(state):
    q, k, v, do = (state[n] for n in ("q", "k", "v", "do"))
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for tq, tk, hq, h, Lq, Lk in _heads(state):
        qh = q[tq, hq].float().transpose(0, 1).contiguous()
        gh = do[tq, hq].float().transpose(0, 1).contiguous()
        kh, vh = k[tk, h].float(), v[tk, h].float()
        p, _ = _softmax(_scores(qh, kh, state["scale"], Lq, Lk))
        dv[tk, h] = torch.matmul(p.reshape(-1, Lk).t(), gh.reshape(-1, gh.shape[-1])).to(dv.dtype)
        dp = torch.matmul(gh, vh.t())
        ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * state["scale"]
        dq[tq, hq] = torch.matmul(ds, kh).transpose(0, 1).to(dq.dtype)
        dk[tk, h] = torch.matmul(ds.reshape(-1, Lk).t(), qh.reshape(-1, qh.shape[-1])).to(dk.dtype)
    return {"dq": dq, "dk": dk, "dv": dv}


def _pow2(e):
    """2^e in fp32, exactly, for an integer tensor e (below -126: 2^-126)."""
    return ((e.clamp(min=-126).to(torch.int32) + 127) << 23).view(torch.float32)


def _exponent(amax):
    """The least integer e with amax <= 448 2^e, kept within EXP_MIN..EXP_MAX (fp32 in, int32 out)."""
    m, x = torch.frexp(amax)  # amax = m 2^x, m in [0.5, 1)
    e = x - 9 + (m > 0.875).to(x.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, EXP_MIN)).clamp_(EXP_MIN, EXP_MAX)


def _append(state):
    block = state["case"]["block"]
    table = state["table"]
    lens, start = state["lens"], state["start"]
    dev = table.device
    # one entry for each block that gets tokens: its page, the tokens it holds already, its first
    # new token and their number
    pages, held, first, count = [], [], [], []
    at = 0
    for n, L in enumerate(lens):
        p, end = start[n], start[n] + L
        while p < end:
            stop = min(end, (p // block + 1) * block)
            pages.append((n, p // block))
            held.append(p % block)
            first.append(at + p - start[n])
            count.append(stop - p)
            p = stop
        at += L
    if not pages:
        return
    idx = torch.tensor(pages, device=dev)
    page = table[idx[:, 0], idx[:, 1]].long()
    held, first, count = (torch.tensor(x, device=dev)[:, None] for x in (held, first, count))
    pos = torch.arange(block, device=dev)[None, :]
    new = (pos >= held) & (pos < held + count)  # [blocks, block]
    old = pos < held
    tok = torch.where(new, first + pos - held, torch.zeros_like(pos))
    for rows, cache, scale, turned in ((state["k"], state["k_cache"], state["k_scale"], False),
                                       (state["v"], state["v_cache"], state["v_scale"], True)):
        x = rows[tok].float() * new[:, :, None, None]  # [blocks, block, Hk, d]
        x = x.transpose(1, 2)
        e = _exponent(x.abs().amax(dim=(2, 3)))  # [blocks, Hk]
        e_old = torch.frexp(scale[page])[1] - 1
        e = torch.where(held > 0, torch.maximum(e, e_old), e)
        b = cache[page].float()
        if turned:
            b = b.transpose(2, 3)
        b = torch.where(old[:, None, :, None], b, torch.zeros_like(b))
        # bytes held already move to the block's new scale; what follows the new tokens is zero
        ee, eo = e[:, :, None, None], e_old[:, :, None, None]
        out = torch.where(new[:, None, :, None], x * _pow2(-ee), b * _pow2(eo - ee))
        if turned:
            out = out.transpose(2, 3)
        cache.view(torch.uint8)[page] = out.to(torch.float8_e4m3fn).view(torch.uint8)
        scale[page] = _pow2(e)


def _decode(state):
    case, q = state["case"], state["q"]
    N, T, H, dk = q.shape
    Hk, dv = case["Hk"], case["dv"]
    G = H // Hk
    o = torch.zeros(N, T, H, dv, dtype=q.dtype, device=q.device)
    for n, L in enumerate(state["lens"]):
        if L == 0:
            continue
        page = state["table"][n, :-(-L // case["block"])].long()
        k = state["k_cache"][page].float() * state["k_scale"][page][:, :, None, None]
        v = state["v_cache"][page].float() * state["v_scale"][page][:, :, None, None]
        k = k.transpose(0, 1).reshape(Hk, -1, dk)[:, :L]
        v = v.permute(1, 0, 3, 2).reshape(Hk, -1, dv)[:, :L]
        for h in range(Hk):
            qh = q[n, :, h * G:h * G + G].float().transpose(0, 1).contiguous()
            p, _ = _softmax(_scores(qh, k[h], state["scale"], T, L))
            o[n, :, h * G:h * G + G] = torch.matmul(p, v[h]).transpose(0, 1).to(o.dtype)
    return o


# ---------------------------------------------------------------------------
# the definitions in fp64
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "decode":
        return _exact_decode(s)
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    G = case["H"] // case["Hk"]
    train = case["op"] == "backward"
    if train:
        do = s["do"].double()
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    o = torch.zeros(*q.shape[:2], v.shape[2], dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    b = 0
    a = 0
    for Lq, Lk in zip(s["lens_q"], s["lens_k"]):
        visible = torch.ones(Lq, Lk, dtype=torch.bool, device=q.device).tril_(Lk - Lq)
        live = visible.any(1) if Lk else torch.zeros(Lq, dtype=torch.bool, device=q.device)
        for h in range(case["H"] if Lq and Lk else 0):
            K, V = k[b:b + Lk, h // G], v[b:b + Lk, h // G]
            Q = q[a:a + Lq, h]
            x = torch.where(visible, Q @ K.T * s["scale"], -math.inf)
            z = torch.logsumexp(x, 1)
            lse[a:a + Lq, h] = z
            P = torch.where(live[:, None], torch.exp(x - torch.where(live, z, 0.0)[:, None]), 0.0)
            O = P @ V
            o[a:a + Lq, h] = O
            if train:
                D = do[a:a + Lq, h]
                dv[b:b + Lk, h // G] += P.T @ D
                dS = P * (D @ V.T - (D * O).sum(1)[:, None])
                dq[a:a + Lq, h] = s["scale"] * (dS @ K)
                dk[b:b + Lk, h // G] += s["scale"] * (dS.T @ Q)
        a, b = a + Lq, b + Lk
    return {"dq": dq, "dk": dk, "dv": dv} if train else {"o": o, "lse": lse}


def _exact_e4m3(y):
    """y (fp64, |y| <= 448) rounded to the nearest e4m3 number, ties to even: 3 fraction bits,
    exponents from -6, steps of 2^-9 below."""
    x = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -30))).clamp_(min=-6)
    step = torch.exp2(x - 3)
    return torch.round(y / step) * step


def _exact_append(s):
    block = s["case"]["block"]
    out = {n: s[n].double() for n in ("k_cache", "v_cache", "k_scale", "v_scale")}
    table = s["table"].tolist()
    at = 0
    for n, L in enumerate(s["lens"]):
        p0 = s["start"][n]
        for b in range(p0 // block, -(-(p0 + L) // block) if L else 0):
            lo, hi = max(p0, b * block), min(p0 + L, (b + 1) * block)
            page, had = table[n][b], max(0, p0 - b * block)
            for rows, c, sc in (("k", "k_cache", "k_scale"), ("v", "v_cache", "v_scale")):
                x = s[rows][at + lo - p0:at + hi - p0].double().transpose(0, 1)  # [Hk, new, d]
                amax = x.abs().amax(dim=(1, 2))
                e = torch.ceil(torch.log2(amax.clamp(min=2.0 ** -200) / E4M3_MAX)).clamp_(EXP_MIN, EXP_MAX)
                body = out[c][page] if c == "k_cache" else out[c][page].transpose(1, 2)
                fresh = torch.zeros_like(body)
                if had:
                    e_old = torch.log2(out[sc][page])
                    e = torch.maximum(e, e_old)
                    fresh[:, :had] = _exact_e4m3(body[:, :had] * torch.exp2(e_old - e)[:, None, None])
                fresh[:, had:had + hi - lo] = _exact_e4m3(x * torch.exp2(-e)[:, None, None])
                out[c][page] = fresh if c == "k_cache" else fresh.transpose(1, 2)
                out[sc][page] = torch.exp2(e)
        at += L
    return out


def _exact_decode(s):
    case, q = s["case"], s["q"].double()
    N, T, H, _ = q.shape
    G = H // case["Hk"]
    o = torch.zeros(N, T, H, case["dv"], dtype=torch.float64, device=q.device)
    for n, L in enumerate(s["lens"]):
        page = s["table"][n, :-(-L // case["block"])].long()
        for h in range(H if L else 0):
            kh = h // G
            K = (s["k_cache"][page, kh].double() * s["k_scale"][page, kh].double()[:, None, None]).flatten(0, 1)[:L]
            V = s["v_cache"][page, kh].double() * s["v_scale"][page, kh].double()[:, None, None]
            V = V.transpose(1, 2).flatten(0, 1)[:L]
            for t in range(T):
                m = L - T + t + 1
                if m > 0:
                    w = torch.softmax(K[:m] @ q[n, t, h] * s["scale"], 0)
                    o[n, t, h] = w @ V[:m]
    return {"o": o}
