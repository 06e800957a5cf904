"""The workloads of the cache-side operators of a verify cycle: ``block_attention`` (the new
tokens of every sequence against its paged cache) and ``rotary_append`` (their rotary
embedding and their append to that cache).

``own`` chooses between the plain form (elementary torch operations in 32 bits) and this
package's kernels. A case fixes every size, the sequence lengths included; the seed makes the
values.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------------------- the cases

def _attention(name, **kw):
    c = dict(name=name, op="attention", B=1, n_lo=1, n_hi=1, len_lo=128, len_hi=128, Hq=32,
             Hkv=8, D=128, page=16, dtype="bf16", causal=True, window=0, packed=False, lse=False,
             lengths=1)
    c.update(kw)
    return c


def _rotary(name, **kw):
    c = dict(name=name, op="rotary", B=1, n_lo=1, n_hi=1, len_lo=128, len_hi=128, Hq=32, Hkv=8,
             D=128, R=128, page=16, dtype="bf16", interleaved=False, theta=500000.0, stretch=1.0,
             magnitude=1.0, lengths=1)
    c.update(kw)
    return c


def listed():
    return [
        # one user, a block of 7 drafts and the anchor on a short context: latency
        _attention("attn_verify_one_user", B=1, n_lo=8, n_hi=8, len_lo=900, len_hi=1100),
        # plain decoding of a serving batch (the requests whose speculation is off)
        _attention("attn_decode_batch", B=64, n_lo=1, n_hi=1, len_lo=256, len_hi=4096, page=64,
                   lengths=2),
        # a mixed serving batch: 0 to 7 drafts and the anchor per sequence
        _attention("attn_verify_serving", B=64, n_lo=1, n_hi=8, len_lo=1024, len_hi=16384,
                   page=64, lengths=3),
        # few long contexts, seven query heads per cache head, the statistics kept for a merge
        _attention("attn_verify_long", B=4, n_lo=8, n_hi=8, len_lo=100000, len_hi=131072, Hq=28,
                   Hkv=4, page=32, dtype="f16", lse=True, lengths=4),
        # a drafter's block: every token of the block sees the whole block and a window
        _attention("attn_draft_block_window", B=32, n_lo=16, n_hi=16, len_lo=2000, len_hi=16000,
                   Hq=16, Hkv=2, D=64, dtype="f16", causal=False, window=4096, lengths=5),
        # chunks of three prompts and the blocks of other requests in one packed call
        _attention("attn_mixed_chunks", B=6, n_lo=5, n_hi=2048, len_lo=2048, len_hi=8192,
                   page=128, packed=True, lengths=6),
        # one large chunk of a long prompt
        _attention("attn_prompt_chunk", B=1, n_lo=4096, n_hi=4096, len_lo=12288, len_hi=12288,
                   page=64, packed=True, lengths=7),
        # one decode step of a small batch
        _rotary("rotary_decode", B=32, n_lo=1, n_hi=1, len_lo=100, len_hi=4096, lengths=8),
        # blocks of a serving batch, half of the head rotated in pairs, a stretched long context
        _rotary("rotary_verify_partial", B=32, n_lo=1, n_hi=8, len_lo=4096, len_hi=65536, Hq=28,
                Hkv=4, R=64, page=32, dtype="f16", interleaved=True, theta=10000.0, stretch=8.0,
                magnitude=1.2079441541679836, lengths=9),
        # chunks of prompts: bandwidth
        _rotary("rotary_prompt", B=4, n_lo=1000, n_hi=4096, len_lo=4096, len_hi=8192, page=64,
                lengths=10),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {op: [max(work(c)[k] for c in listed() if c["op"] == op) for k in ("bytes", "flops")]
            for op in ("attention", "rotary")}
    while True:
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        common = dict(B=_log_int(rng, 1, 64), Hkv=Hkv, Hq=Hkv * rng.choice([1, 2, 4, 5, 7, 8]),
                      D=D, page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["bf16", "f16"]),
                      lengths=rng.randrange(1 << 30))
        if rng.random() < 0.65:
            n = _log_int(rng, 1, 4096) if rng.random() < 0.5 else rng.randint(1, 16)
            lo = _log_int(rng, max(n, 64), 65536)
            c = _attention("", n_lo=max(1, n // rng.choice([1, 1, 3])), n_hi=n, len_lo=lo,
                           len_hi=_log_int(rng, lo, 131072), causal=rng.random() < 0.8,
                           window=rng.choice([0, 0, 0, 512, 4096]), packed=rng.random() < 0.5,
                           lse=rng.random() < 0.3, **common)
        else:
            n = _log_int(rng, 1, 4096)
            lo = _log_int(rng, n, 65536)
            c = _rotary("", n_lo=max(1, n // 3), n_hi=n, len_lo=lo,
                        len_hi=_log_int(rng, lo, 131072), R=rng.choice([D, D // 2, D // 4]),
                        interleaved=rng.random() < 0.5, theta=rng.choice([1e4, 5e5]),
                        stretch=rng.choice([1.0, 4.0]), **common)
        del c["name"]
        # the plain form pads every sequence to the longest one and keeps every score
        n_new, kv_len = _lengths(c)
        pad = c["B"] * max(kv_len)
        scores = pad * max(n_new) * c["Hq"] if c["op"] == "attention" else 0
        w = work(c)
        if pad * c["Hkv"] * D <= 1 << 30 and scores <= 1 << 31 and \
                w["bytes"] <= most[c["op"]][0] and w["flops"] <= most[c["op"]][1]:
            return c


def _lengths(c):
    """The new tokens and the cache length (the new tokens included) of every sequence."""
    rng = random.Random(c["lengths"])
    n_new = [rng.randint(c["n_lo"], c["n_hi"]) for _ in range(c["B"])]
    kv_len = [max(n, _log_int(rng, c["len_lo"], c["len_hi"])) for n in n_new]
    return n_new, kv_len


def work(c):
    n_new, kv_len = _lengths(c)
    T, es = sum(n_new), 2
    if c["op"] == "rotary":
        row = (c["Hq"] + 2 * c["Hkv"]) * c["D"] * es
        return {"bytes": 2 * T * row + 2 * c["R"] + 8 * c["B"] + 4 * T,
                "flops": 3 * T * (c["Hq"] + c["Hkv"]) * c["R"]}
    seen = pairs = 0
    for n, L in zip(n_new, kv_len):
        first = max(0, L - n - c["window"] + 1) if c["window"] else 0
        seen += L - first
        if c["causal"] and not c["window"]:
            pairs += n * (L - n) + n * (n + 1) // 2
        else:
            for p in range(L - n, L):
                hi = p + 1 if c["causal"] else L
                pairs += hi - (max(0, p - c["window"] + 1) if c["window"] else 0)
    pages = sum(-(-L // c["page"]) for L in kv_len)
    return {"bytes": 2 * T * c["Hq"] * c["D"] * es + 2 * seen * c["Hkv"] * c["D"] * es +
            4 * pages + 8 * c["B"] + (4 * T * c["Hq"] if c["lse"] else 0),
            "flops": 4 * c["D"] * c["Hq"] * pairs}


# ------------------------------------------------------------------------------- the inputs

def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    n_new, kv_len = _lengths(c)
    B, ps, Hkv, D = c["B"], c["page"], c["Hkv"], c["D"]
    # a pool of pages in random order, a few of them free
    count = [-(-L // ps) for L in kv_len]
    n_pages = sum(count) + 3
    order = torch.randperm(n_pages, generator=g, device=dev, dtype=torch.int32)
    start = torch.tensor([sum(count[:b]) for b in range(B)], device=dev)
    col = torch.arange(max(count), device=dev)
    have = col[None, :] < torch.tensor(count, device=dev)[:, None]
    table = torch.where(have, order[(start[:, None] + col[None, :]).clamp(max=n_pages - 1)], 0)
    s = {"case": c, "page_table": table.to(torch.int32).contiguous(),
         "kv_len": torch.tensor(kv_len, dtype=torch.int32, device=dev)}
    shape = (n_pages, ps, Hkv, D)
    T = sum(n_new)
    starts = torch.tensor([sum(n_new[:b]) for b in range(B + 1)], dtype=torch.int32, device=dev)
    if c["op"] == "rotary":
        s["q_start"] = starts
        s["q"] = torch.randn(T, c["Hq"], D, generator=g, device=dev, dtype=dt)
        s["k"] = torch.randn(T, Hkv, D, generator=g, device=dev, dtype=dt)
        s["v"] = torch.randn(T, Hkv, D, generator=g, device=dev, dtype=dt)
        s["k_pages"] = torch.zeros(shape, device=dev, dtype=dt)
        s["v_pages"] = torch.zeros(shape, device=dev, dtype=dt)
        i = torch.arange(0, c["R"], 2, dtype=torch.float64, device=dev)
        s["inv_freq"] = (c["theta"] ** (-i / c["R"]) / c["stretch"]).float()
        s["out"] = torch.empty_like(s["q"])
        return s
    s["k_pages"] = torch.randn(shape, generator=g, device=dev, dtype=dt)
    s["v_pages"] = torch.randn(shape, generator=g, device=dev, dtype=dt)
    lead = (T,) if c["packed"] else (B, c["n_hi"])
    # queries of about twice the keys' size: a few keys stand out, as in a trained head
    s["q"] = 2 * torch.randn(*lead, c["Hq"], D, generator=g, device=dev, dtype=dt)
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros(*lead, c["Hq"], device=dev) if c["lse"] else None
    s["q_start"] = starts if c["packed"] else None
    s["n_new"] = None if c["packed"] else torch.tensor(n_new, dtype=torch.int32, device=dev)
    s["n_max"] = max(n_new)
    return s


# ------------------------------------------------------------------------------- a pass

def run(s):
    if own:
        import lossless_draft_verification_speculative_b200 as dv

        c = s["case"]
        if c["op"] == "rotary":
            q = dv.rotary_append(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"],
                                 s["page_table"], s["kv_len"], s["inv_freq"],
                                 q_start=s["q_start"], interleaved=c["interleaved"],
                                 magnitude=c["magnitude"], out=s["out"])
            return q, s["k_pages"], s["v_pages"]
        out = dv.block_attention(s["q"], s["k_pages"], s["v_pages"], s["page_table"],
                                 s["kv_len"], n_new=s["n_new"], q_start=s["q_start"],
                                 causal=c["causal"], window=c["window"] or None, out=s["out"],
                                 lse=s["lse"])
        return (out, s["lse"]) if c["lse"] else out
    return _rotary_plain(s) if s["case"]["op"] == "rotary" else _attention_plain(s)


def _token_places(q_start, T):
    """The sequence of every packed token and the token's index in it."""
    t = torch.arange(T, device=q_start.device)
    b = torch.searchsorted(q_start[1:].long(), t, right=True)
    return b, t - q_start.long()[b]


def _rotary_plain(s):
    c = s["case"]
    T = s["q"].shape[0]
    b, i = _token_places(s["q_start"], T)
    n = (s["q_start"][1:] - s["q_start"][:-1]).long()
    pos = s["kv_len"].long()[b] - n[b] + i
    angle = pos.double()[:, None] * s["inv_freq"].double()[None, :]
    cos = (c["magnitude"] * torch.cos(angle)).float()[:, None, :]
    sin = (c["magnitude"] * torch.sin(angle)).float()[:, None, :]

    def turn(x):
        x = x.float()
        R = c["R"]
        y = x.clone()
        first, second = (slice(0, R, 2), slice(1, R, 2)) if c["interleaved"] else \
            (slice(0, R // 2), slice(R // 2, R))
        a, d = x[..., first], x[..., second]
        y[..., first] = a * cos - d * sin
        y[..., second] = d * cos + a * sin
        return y.to(s["q"].dtype)

    page = s["page_table"].long()[b, pos // c["page"]]
    s["k_pages"][page, pos % c["page"]] = turn(s["k"])
    s["v_pages"][page, pos % c["page"]] = s["v"]
    return turn(s["q"]), s["k_pages"], s["v_pages"]


def _attention_plain(s):
    c = s["case"]
    B, N, Hq, Hkv, D = c["B"], s["n_max"], c["Hq"], c["Hkv"], c["D"]
    G, dev = Hq // Hkv, s["q"].device
    kv_len = s["kv_len"].long()
    if c["packed"]:
        first = s["q_start"].long()
        n_new = first[1:] - first[:-1]
        rows = (first[:-1, None] + torch.arange(N, device=dev)).clamp(max=s["q"].shape[0] - 1)
        q = s["q"][rows].float()
    else:
        n_new = s["n_new"].long()
        q = s["q"][:, :N].float()
    pos = torch.arange(s["page_table"].shape[1] * c["page"], device=dev)
    page = s["page_table"].long()[:, pos // c["page"]]
    slot = (pos % c["page"])[None, :]
    live = pos[None, :] < kv_len[:, None]
    k = s["k_pages"][page, slot].float()
    v = s["v_pages"][page, slot].float().masked_fill_(~live[:, :, None, None], 0.0)
    q = q.view(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D)
    z = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(D))
    place = (kv_len - n_new)[:, None] + torch.arange(N, device=dev)
    seen = live[:, None, :].expand(B, N, pos.numel())
    if c["causal"]:
        seen = seen & (pos <= place[:, :, None])
    if c["window"]:
        seen = seen & (pos > place[:, :, None] - c["window"])
    z = z.view(B, Hkv, N, G, -1).masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = z.amax(-1, keepdim=True).clamp_(min=-3e38)
    z = z.sub_(m).exp_()
    total = z.sum(-1, keepdim=True)
    o = torch.matmul(z.view(B, Hkv, N * G, -1), v.permute(0, 2, 1, 3)).view(B, Hkv, N, G, D)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D)
    lse = (m + torch.log(total))[..., 0].permute(0, 2, 1, 3).reshape(B, N, Hq)
    if c["packed"]:
        b, i = _token_places(s["q_start"], s["q"].shape[0])
        out, stat = o[b, i], lse[b, i]
    else:
        real = torch.arange(N, device=dev)[None, :] < n_new[:, None]
        out = s["out"].clone()
        out[:, :N] = torch.where(real[:, :, None, None], o.to(out.dtype), out[:, :N])
        stat = torch.zeros(B, c["n_hi"], Hq, device=dev)
        stat[:, :N] = torch.where(real[:, :, None], lse, 0.0)
    out = out.to(s["q"].dtype)
    return (out, stat) if c["lse"] else out


# ------------------------------------------------------------------------------- 64 bits

def exact(c, seed):
    s = prepare(c, seed)
    n_new, kv_len = _lengths(c)
    ps, Hkv, D, G = c["page"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"]
    if c["op"] == "rotary":
        k_pages, v_pages, qs, t = s["k_pages"].double(), s["v_pages"].double(), [], 0
        half = c["R"] // 2
        for b in range(c["B"]):
            n, L = n_new[b], kv_len[b]
            where = torch.arange(L - n, L, device="cuda")
            phase = where.double()[:, None] * s["inv_freq"].double()[None, :]
            # a pair is a complex number, turned by exp(i phase)
            spin = torch.polar(torch.full_like(phase, c["magnitude"]), phase)[:, None, :]
            made = {}
            for key in ("q", "k"):
                x = s[key][t:t + n].double()
                head, rest = x[..., :c["R"]], x[..., c["R"]:]
                if c["interleaved"]:
                    z = torch.view_as_complex(head.reshape(*head.shape[:-1], half, 2).contiguous())
                    head = torch.view_as_real(z * spin).reshape(head.shape)
                else:
                    z = torch.complex(head[..., :half], head[..., half:]) * spin
                    head = torch.cat([z.real, z.imag], -1)
                made[key] = torch.cat([head, rest], -1)
            qs.append(made["q"])
            flat = s["page_table"][b].long()[where // ps] * ps + where % ps
            k_pages.view(-1, Hkv, D)[flat] = made["k"]
            v_pages.view(-1, Hkv, D)[flat] = s["v"][t:t + n].double()
            t += n
        return torch.cat(qs), k_pages, v_pages
    if work(c)["flops"] > 2e12:
        return None
    out, stat = s["out"].double(), torch.zeros(s["q"].shape[:-1], device="cuda").double()
    t = 0
    for b in range(c["B"]):
        n, L = n_new[b], kv_len[b]
        at = (slice(t, t + n),) if c["packed"] else (b, slice(0, n))
        t += n
        pages = s["page_table"][b, :-(-L // ps)].long()
        K = s["k_pages"][pages].reshape(-1, Hkv, D)[:L]
        V = s["v_pages"][pages].reshape(-1, Hkv, D)[:L]
        key, mine = torch.arange(L, device="cuda"), torch.arange(L - n, L, device="cuda")
        hide = torch.zeros(n, L, dtype=torch.bool, device="cuda")
        if c["causal"]:
            hide |= key[None, :] > mine[:, None]
        if c["window"]:
            hide |= key[None, :] <= mine[:, None] - c["window"]
        q = s["q"][at]
        o, z = out[at], stat[at]
        for h in range(c["Hq"]):
            score = q[:, h].double() @ K[:, h // G].double().T / math.sqrt(D)
            score.masked_fill_(hide, -math.inf)
            z[:, h] = torch.logsumexp(score, -1)
            o[:, h] = torch.exp(score - z[:, h, None]) @ V[:, h // G].double()
    return (out, stat) if c["lse"] else out
