"""Workloads of the decode-step operators around the quantized products: the
paged key-value cache (rotate and store, read back), the attention of one new
token over it, and the adjustment of logits before sampling.

``run`` takes the plain form (elementary torch operations in 32 bits) where
``own`` is false and the library's calls where it is true; ``exact`` gives the
same outputs in 64 bits.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # One user, a short chat: the latency of a single small call.
        attend("attend one short", 1, 337, 8, 4, 128, "bf16", 16, "f32"),
        # A continuous batch of ordinary lengths, one slot of it empty and one just begun.
        attend("attend batch 16", 16, 4001, 8, 4, 128, "bf16", 16, "f32"),
        # A full server with the cache in 8 bits: the largest read.
        attend("attend batch 64 q8_0", 64, 16384, 8, 4, 128, "q8_0", 32, "f32"),
        # One long document, capped scores, wide groups.
        attend("attend one long capped", 1, 131071, 4, 8, 128, "f16", 64, "bf16", softcap=50.0),
        # Heads of their own, a sliding window, biases by distance, pages of an odd size.
        attend("attend windows alibi", 24, 3001, 12, 1, 64, "f16", 24, "f32", window=1024,
               alibi=True),
        # The step of a small batch: one token of each sequence.
        append("append batch 16", 16, 8, 4, 128, "bf16", 16, "f32"),
        # The prompt of a picture and its text: three position axes.
        append("append prompt 3 axes", 4096, 8, 4, 128, "f16", 32, "bf16", axes=3),
        # A prompt into the 8-bit cache, and its values read back.
        append("append prompt q8_0", 2011, 8, 4, 128, "q8_0", 32, "f32"),
        # The cached prefix of one sequence taken out of the 8-bit cache.
        read("read prefix q8_0", 16384, 8, 128, "q8_0", 32, "bf16"),
        # A few hundred tokens, 32-bit values wanted.
        read("read short", 301, 8, 64, "bf16", 16, "f32"),
        # One row of logits with everything on.
        logits("logits one", 1, 128256, "f32", 700, 20, True),
        # A large batch.
        logits("logits batch 256", 256, 128256, "f32", 2000, 100, True),
    ]


def attend(name, B, L, kv_heads, group, D, cache, page, io, softcap=0.0, window=0, alibi=False):
    return {"name": name, "op": "attend", "B": B, "L": L, "kv_heads": kv_heads, "group": group,
            "D": D, "cache": cache, "page": page, "io": io, "softcap": softcap, "window": window,
            "alibi": alibi}


def append(name, T, kv_heads, group, D, cache, page, io, axes=1, pairing="halves", n_rot=0):
    return {"name": name, "op": "append", "T": T, "kv_heads": kv_heads, "group": group, "D": D,
            "cache": cache, "page": page, "io": io, "axes": axes, "pairing": pairing,
            "n_rot": n_rot or D}


def read(name, T, kv_heads, D, cache, page, io):
    return {"name": name, "op": "read", "T": T, "kv_heads": kv_heads, "D": D, "cache": cache,
            "page": page, "io": io}


def logits(name, B, V, io, history, biases, masked):
    return {"name": name, "op": "logits", "B": B, "V": V, "io": io, "history": history,
            "biases": biases, "masked": masked}


def _between(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "read", "logits"])
    D = rng.choice([64, 64, 96, 128, 128, 128, 192, 256])
    cache = rng.choice(["f16", "bf16", "q8_0"])
    page = rng.choice([1, 8, 16, 16, 24, 32, 64, 100, 256])
    io = rng.choice(["f32", "f32", "f16", "bf16"])
    kv_heads = rng.choice([1, 2, 3, 4, 8, 8, 16])
    if op == "attend":
        B = _between(rng, 1, 128)
        cells = 64 * 16384 * 8 * 128 // 2  # keys' values, at most half the largest case's
        most = max(16, min(131071, cells // (B * kv_heads * D)))
        L = _between(rng, 1, most)
        c = attend("", B, L, kv_heads, rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16]), D, cache, page,
                   io, softcap=rng.choice([0.0, 0.0, 30.0, 50.0]),
                   window=rng.choice([0, 0, 0, 127, 1000, 4096]), alibi=rng.random() < 0.25)
    elif op == "append":
        T = _between(rng, 1, 4096)
        c = append("", T, min(kv_heads, 8), rng.choice([1, 2, 4, 7]), D, cache, page, io,
                   axes=rng.choice([1, 1, 2, 3, 4]), pairing=rng.choice(["halves", "adjacent"]),
                   n_rot=rng.choice([D, D, D // 2, D // 4]))
    elif op == "read":
        c = read("", _between(rng, 1, 16384), min(kv_heads, 8), D, cache, page, io)
    else:
        B = _between(rng, 1, 128)
        c = logits("", B, _between(rng, 1000, 262144), io, rng.choice([0, 33, 500, 2000]),
                   rng.choice([0, 1, 20, 300]), rng.random() < 0.6)
    del c["name"]
    return c


# ------------------------------------------------------------------ what a pass cannot do without

def _row_bytes(case):
    """Bytes of one head's row in the cache."""
    D = case["D"]
    return D * 34 // 32 if case["cache"] == "q8_0" else 2 * D


def _lens(case):
    """Lengths from half the longest up; in a batch one sequence is empty and one has just begun."""
    B, L = case["B"], case["L"]
    out = [L - (i * 7919) % (L // 2 + 1) for i in range(B)]
    if B >= 4:
        out[1], out[2] = 0, 1
    return out


def work(case):
    op, e = case["op"], SIZES[case["io"]]
    if op == "attend":
        rows = case["kv_heads"] * case["group"]
        keys = sum(min(n, case["window"]) if case["window"] else n for n in _lens(case))
        io = case["B"] * rows * (2 * case["D"] * e + 4)
        pages = sum(-(-n // case["page"]) for n in _lens(case)) * 4
        return {"bytes": keys * case["kv_heads"] * 2 * _row_bytes(case) + io + pages,
                "flops": 4 * keys * rows * case["D"]}
    if op == "append":
        T, H, D = case["T"], case["kv_heads"], case["D"]
        nq = H * case["group"]
        n = T * (nq + 2 * H) * D * e + T * nq * D * e + T * 2 * H * _row_bytes(case) + 12 * T
        if case["cache"] == "q8_0":  # and read back in 16 bits
            n += T * 2 * H * (_row_bytes(case) + 2 * D)
        return {"bytes": n, "flops": 3 * T * (nq + H) * case["n_rot"]}
    if op == "read":
        T, H = case["T"], case["kv_heads"]
        return {"bytes": T * 2 * H * (_row_bytes(case) + case["D"] * e) + 8 * T, "flops": 0}
    B, V = case["B"], case["V"]
    n = 2 * B * V * e + B * (4 * case["history"] + 8 * case["biases"])
    return {"bytes": n + (B * ((V + 31) // 32) * 4 if case["masked"] else 0), "flops": 4 * B * V}


# ------------------------------------------------------------------ inputs

def _cache_buffers(case, n_pages, gen):
    """The cache's two buffers with stale values in every slot, and views of what they hold."""
    H, S, D = case["kv_heads"], case["page"], case["D"]
    made = []
    for _ in range(2):
        if case["cache"] == "q8_0":
            n, sc = n_pages * H * S * D, (D // 32 + 1) // 2 * 2
            buf = torch.empty(n + n_pages * H * S * sc * 2, dtype=torch.uint8, device="cuda")
            codes = buf[:n].view(torch.int8).view(n_pages, H, S, D)
            scales = buf[n:].view(torch.float16).view(n_pages, H, S, sc)
            codes.random_(-127, 128, generator=gen)
            scales.uniform_(0.005, 0.02, generator=gen)
            made.append((buf, codes, scales))
        else:
            buf = torch.empty(n_pages, H, S, D, dtype=DTYPES[case["cache"]], device="cuda")
            buf.normal_(generator=gen)
            made.append((buf, buf, None))
    return made


def _handle(case, st, n_pages):
    if own:
        import quantized_gguf_dequant_gb300 as q
        kind = {"f16": q.F16, "bf16": q.BF16, "q8_0": q.Q8_0}[case["cache"]]
        st["handle"] = q.KVCache(kind, n_pages, case["page"], case["kv_heads"], case["D"],
                                 k=st["k"][0], v=st["v"][0])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    order = random.Random(seed)
    st = {"case": case}
    io = DTYPES[case["io"]]

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen).to(io)

    if case["op"] == "attend":
        lens, S = _lens(case), case["page"]
        order.shuffle(lens)
        need = [-(-n // S) for n in lens]
        n_pages = sum(need) + 3
        free = np.random.RandomState(seed % (1 << 31)).permutation(n_pages)
        table = np.full((case["B"], max(need)), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = free[at:at + n]
            at += n
        rows = case["kv_heads"] * case["group"]
        st["k"], st["v"] = _cache_buffers(case, n_pages, gen)
        st["q"] = normal(case["B"], rows, case["D"])
        st["table"] = torch.from_numpy(table).cuda()
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st["longest"] = max(lens)
        st["scale"] = 1.0 / math.sqrt(case["D"])
        st["alibi"] = None
        if case["alibi"]:
            st["alibi"] = torch.exp2(-8.0 * (torch.arange(rows, device="cuda") + 1) / rows)
        _handle(case, st, n_pages)
    elif case["op"] == "append":
        T, S, H, D = case["T"], case["page"], case["kv_heads"], case["D"]
        nq = H * case["group"]
        qkv = normal(T, nq + 2 * H, D)  # the fused projection's output: q, k and v are slices
        st["q"], st["new_k"], st["new_v"] = qkv.split([nq, H, H], dim=1)
        single = T <= 64  # tokens of as many sequences, else one sequence's prompt
        n_pages = (T if single else -(-T // S)) + 5
        pages = torch.randperm(n_pages, device="cuda", generator=gen)
        t = torch.arange(T, device="cuda")
        st["slots"] = pages[t] * S + t * 5 % S if single else pages[t // S] * S + t % S
        if single and T >= 4:
            st["slots"][3] = -1  # a padded row of the batch
        if single:
            first = torch.randint(0, 131072, (T,), device="cuda", generator=gen)
            pos = torch.stack([first + 3 * a for a in range(case["axes"])])
        else:  # text counts on, a picture's rows and columns run within it
            pos = torch.stack([t if a == 0 else 17 + (t // 64 if a == 1 else t % 64)
                               for a in range(case["axes"])])
        st["pos"] = pos.to(torch.int32).contiguous()
        half = case["n_rot"] // 2
        st["inv_freq"] = 500000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float32)
                                      / half)
        cut = [half * (a + 1) // case["axes"] for a in range(case["axes"])]
        st["sections"] = [c - p for c, p in zip(cut, [0] + cut)]
        axis = np.repeat(np.arange(case["axes"]), st["sections"])
        st["axis"] = torch.from_numpy(axis).cuda()
        st["k"], st["v"] = _cache_buffers(case, n_pages, gen)
        _handle(case, st, n_pages)
        if own:
            import quantized_gguf_dequant_gb300 as q
            st["rope"] = q.Rope(st["inv_freq"], st["sections"], pairing=case["pairing"])
    elif case["op"] == "read":
        T, S = case["T"], case["page"]
        n_pages = -(-T // S) + 5
        pages = torch.randperm(n_pages, device="cuda", generator=gen)
        t = torch.arange(T, device="cuda")
        st["slots"] = pages[t // S] * S + t % S
        st["k"], st["v"] = _cache_buffers(case, n_pages, gen)
        _handle(case, st, n_pages)
    else:
        B, V = case["B"], case["V"]
        st["logits"] = (3 * torch.randn(B, V, device="cuda", generator=gen)).to(io)
        lens = [case["history"] - (b * 7919) % (case["history"] // 2 + 1) for b in range(B)]
        order.shuffle(lens)
        n = sum(lens)
        u = torch.rand(n, device="cuda", generator=gen)
        ids = (u.pow(3) * V).to(torch.int32)  # some tokens are frequent, most are not
        ids[::97] = -1  # padding
        st["history"], st["n_history"] = ids, n
        st["history_offsets"] = _offsets(lens)
        for name, lo, hi in (("repeat", 1.0, 1.3), ("presence", 0.0, 0.6), ("frequency", 0.0, 0.3)):
            st[name] = lo + (hi - lo) * torch.rand(B, device="cuda", generator=gen)
        each = min(case["biases"], V)
        at = torch.randint(0, V, (B, 1), device="cuda", generator=gen)
        stride = max(1, V // max(1, each))
        st["bias_ids"] = ((at + stride * torch.arange(each, device="cuda")) % V).to(torch.int32).view(-1)
        st["bias_values"] = 4 * torch.randn(B * each, device="cuda", generator=gen)
        st["bias_offsets"] = _offsets([each] * B)
        st["mask"] = None
        if case["masked"]:
            st["mask"] = torch.randint(-(1 << 31), 1 << 31, (B, (V + 31) // 32), device="cuda",
                                       generator=gen).to(torch.int32)
            if B >= 4:
                st["mask"][1] = 0  # a grammar that has ended: nothing is allowed
    return st


def _offsets(lens):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)).cuda()


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"attend": _own_attend, "append": _own_append, "read": _own_read,
                "logits": _own_logits}[op](state)
    return {"attend": _attend, "append": _append, "read": _read, "logits": _logits}[op](state)


def _own_attend(st):
    c = st["case"]
    out, lse = st["handle"].attend(st["q"], st["table"], st["lens"], scale=st["scale"],
                                   softcap=c["softcap"], window=c["window"], alibi=st["alibi"],
                                   return_lse=True)
    return {"out": out, "lse": lse}


def _own_append(st):
    c = st["case"]
    q = st["handle"].append(st["new_k"], st["new_v"], st["slots"], q=st["q"], pos=st["pos"],
                            rope=st["rope"])
    if c["cache"] == "q8_0":
        k, v = st["handle"].read(st["slots"], torch.bfloat16)
        return {"q": q, "k": k, "v": v}
    return {"q": q, "k": st["k"][0], "v": st["v"][0]}


def _own_read(st):
    k, v = st["handle"].read(st["slots"], DTYPES[st["case"]["io"]])
    return {"k": k, "v": v}


def _own_logits(st):
    import quantized_gguf_dequant_gb300 as q
    return {"logits": q.logits_adjust(
        st["logits"], history=st["history"], history_offsets=st["history_offsets"],
        repeat=st["repeat"], presence=st["presence"], frequency=st["frequency"],
        bias_ids=st["bias_ids"], bias_values=st["bias_values"], bias_offsets=st["bias_offsets"],
        mask=st["mask"])}


def _values(part, page, offset):
    """The fp32 values of the cache's rows at (page, offset): [..., heads, D]."""
    _, held, scales = part
    x = held[page, :, offset].float()
    if scales is not None:
        d = scales[page, :, offset].float()[..., :x.shape[-1] // 32]
        x = (x.unflatten(-1, (-1, 32)) * d.unsqueeze(-1)).flatten(-2)
    return x


def _attend(st):
    c = st["case"]
    B, H, G, D, S = c["B"], c["kv_heads"], c["group"], c["D"], c["page"]
    j = torch.arange(st["longest"], device="cuda")
    page = st["table"][:, j // S].clamp(min=0).long()
    k = _values(st["k"], page, j % S)
    q = st["q"].float().view(B, H, G, D)
    s = torch.matmul(q, k.permute(0, 2, 3, 1)) * st["scale"]
    del k
    if c["softcap"]:
        s = c["softcap"] * torch.tanh(s / c["softcap"])
    n = st["lens"].long().view(B, 1)
    if st["alibi"] is not None:
        s = s + st["alibi"].view(1, H, G, 1) * (j - (n - 1)).float().view(B, 1, 1, -1)
    seen = j < n
    if c["window"]:
        seen = seen & (j >= n - c["window"])
    s = torch.where(seen.view(B, 1, 1, -1), s, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    v = _values(st["v"], page, j % S)
    out = torch.matmul(p, v.transpose(1, 2)) / torch.where(total > 0, total, 1.0)
    lse = (m + torch.log(total)).view(B, H * G)
    return {"out": out.view(B, H * G, D).to(st["q"].dtype), "lse": lse}


def _rotated(st, x):
    c = st["case"]
    n, half = c["n_rot"], c["n_rot"] // 2
    angle = (st["pos"].float()[st["axis"]] * st["inv_freq"].unsqueeze(1)).t().unsqueeze(1)
    cos, sin = torch.cos(angle), torch.sin(angle)
    x = x.float()
    if c["pairing"] == "halves":
        a, b = x[..., :half], x[..., half:n]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = x[..., 0:n:2], x[..., 1:n:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([turned, x[..., n:]], dim=-1)


def _store(part, x, page, offset):
    _, held, scales = part
    if scales is None:
        held[page, :, offset] = x.to(held.dtype)
        return
    blocks = x.unflatten(-1, (-1, 32))
    d = blocks.abs().amax(-1, keepdim=True) / 127.0
    inv = torch.where(d > 0, 1.0 / d, 0.0)
    held[page, :, offset] = torch.round(blocks * inv).flatten(-2).to(torch.int8)
    scales[page, :, offset, :d.shape[-2]] = d.squeeze(-1).half()


def _append(st):
    c = st["case"]
    q = _rotated(st, st["q"]).to(st["q"].dtype)
    k = _rotated(st, st["new_k"])
    slots = st["slots"]
    kept = slots >= 0
    page, offset = slots[kept] // c["page"], slots[kept] % c["page"]
    _store(st["k"], k[kept], page, offset)
    _store(st["v"], st["new_v"].float()[kept], page, offset)
    if c["cache"] == "q8_0":
        return {"q": q, **_take(st, torch.bfloat16)}
    return {"q": q, "k": st["k"][0], "v": st["v"][0]}


def _take(st, dtype):
    slots, S = st["slots"], st["case"]["page"]
    kept = (slots >= 0).view(-1, 1, 1)
    page, offset = slots.clamp(min=0) // S, slots.clamp(min=0) % S
    return {n: torch.where(kept, _values(st[n], page, offset), 0.0).to(dtype) for n in ("k", "v")}


def _read(st):
    return _take(st, DTYPES[st["case"]["io"]])


def _counts(st, rows, ids, values, dtype):
    """values summed by (row, id); ids outside the vocabulary are left out."""
    B, V = st["case"]["B"], st["case"]["V"]
    ids = ids.long()
    at = torch.where((ids >= 0) & (ids < V), rows * V + ids, B * V)
    return torch.zeros(B * V + 1, device="cuda", dtype=dtype).index_add_(
        0, at, values)[:B * V].view(B, V)


def _rows_of(st, offsets, n):
    b = torch.arange(st["case"]["B"], device="cuda")
    return torch.repeat_interleave(b, offsets[1:] - offsets[:-1], output_size=n)


def _adjusted(st, dtype):
    z = st["logits"].to(dtype)
    n = st["n_history"]
    count = _counts(st, _rows_of(st, st["history_offsets"], n), st["history"],
                    torch.ones(n, device="cuda", dtype=dtype), dtype)
    r, pres, freq = (st[k].to(dtype).unsqueeze(1) for k in ("repeat", "presence", "frequency"))
    hit = torch.where(z > 0, z / r, z * r) - (pres + freq * count)
    z = torch.where(count > 0, hit, z)
    n = st["bias_ids"].numel()
    z = z + _counts(st, _rows_of(st, st["bias_offsets"], n), st["bias_ids"],
                    st["bias_values"].to(dtype), dtype)
    if st["mask"] is not None:
        v = torch.arange(st["case"]["V"], device="cuda")
        allowed = (st["mask"][:, v // 32] >> (v % 32)) & 1
        z = torch.where(allowed != 0, z, -math.inf)
    return z


def _logits(st):
    return {"logits": _adjusted(st, torch.float32).to(st["logits"].dtype)}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"attend": _exact_attend, "append": _exact_append, "read": _exact_read,
            "logits": _exact_logits}[case["op"]](st)


def _doubles(part, page, offset):
    _, held, scales = part
    x = held[page, :, offset].double()
    if scales is not None:
        d = scales[page, :, offset].double()[..., :x.shape[-1] // 32]
        x = x * torch.repeat_interleave(d, 32, dim=-1)
    return x


def _exact_attend(st):
    c = st["case"]
    H, G, D, S = c["kv_heads"], c["group"], c["D"], c["page"]
    out = torch.zeros(c["B"], H * G, D, dtype=torch.float64, device="cuda")
    lse = torch.full((c["B"], H * G), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(st["lens"].tolist()):
        first = max(0, n - c["window"]) if c["window"] else 0
        if n == first:
            continue
        j = torch.arange(first, n, device="cuda")
        page = st["table"][b].long()[j // S]
        k, v = _doubles(st["k"], page, j % S), _doubles(st["v"], page, j % S)
        for h in range(H * G):
            s = k[:, h // G] @ st["q"][b, h].double() * st["scale"]
            if c["softcap"]:
                s = c["softcap"] * torch.tanh(s / c["softcap"])
            if st["alibi"] is not None:
                s = s + st["alibi"][h].double() * (j - (n - 1))
            lse[b, h] = torch.logsumexp(s, 0)
            out[b, h] = torch.softmax(s, 0) @ v[:, h // G]
    return {"out": out, "lse": lse}


def _exact_append(st):
    c = st["case"]
    T, n, S = c["T"], c["n_rot"], c["page"]
    # the angle is defined as one 32-bit product; what follows is in 64 bits
    pos, inv = st["pos"].cpu().numpy().astype(np.float32), st["inv_freq"].cpu().numpy()
    axis = st["axis"].cpu().numpy()
    angle = np.stack([pos[axis[i]] * inv[i] for i in range(n // 2)], axis=1).astype(np.float64)
    turn = np.exp(1j * angle)[:, None, :]

    def rotate(x):
        x = x.double().cpu().numpy().copy()
        lo = np.arange(n // 2) if c["pairing"] == "halves" else 2 * np.arange(n // 2)
        hi = lo + n // 2 if c["pairing"] == "halves" else lo + 1
        z = (x[..., lo] + 1j * x[..., hi]) * turn
        x[..., lo], x[..., hi] = z.real, z.imag
        return x

    made = {"q": torch.from_numpy(rotate(st["q"]))}
    slots = st["slots"].cpu().numpy()
    rows = {"k": rotate(st["new_k"]), "v": st["new_v"].double().cpu().numpy()}
    for name, x in rows.items():
        if c["cache"] == "q8_0":
            b = x.reshape(T, x.shape[1], -1, 32)
            d = np.abs(b).max(-1, keepdims=True) / 127
            codes = np.rint(np.divide(b, d, out=np.zeros_like(b), where=d > 0))
            x = (codes * d.astype(np.float16).astype(np.float64)).reshape(x.shape)
            x[slots < 0] = 0
            made[name] = torch.from_numpy(x)
        else:
            held = st[name][0].double().cpu().numpy()
            for t in np.nonzero(slots >= 0)[0]:
                held[slots[t] // S, :, slots[t] % S] = x[t]
            made[name] = torch.from_numpy(held)
    return made


def _exact_read(st):
    S = st["case"]["page"]
    page, offset = st["slots"] // S, st["slots"] % S
    return {n: _doubles(st[n], page, offset) for n in ("k", "v")}


def _exact_logits(st):
    c = st["case"]
    z = st["logits"].double().cpu().numpy()
    history, biases = st["history"].cpu().numpy(), st["bias_values"].double().cpu().numpy()
    ids, mask = st["bias_ids"].cpu().numpy(), st["mask"]
    h_at, b_at = st["history_offsets"].tolist(), st["bias_offsets"].tolist()
    par = [st[k].double().cpu().numpy() for k in ("repeat", "presence", "frequency")]
    for b in range(c["B"]):
        said = history[h_at[b]:h_at[b + 1]]
        tokens, count = np.unique(said[(said >= 0) & (said < c["V"])], return_counts=True)
        x = z[b, tokens]
        x = np.where(x > 0, x / par[0][b], x * par[0][b])
        z[b, tokens] = x - (par[1][b] + par[2][b] * count)
        np.add.at(z[b], ids[b_at[b]:b_at[b + 1]], biases[b_at[b]:b_at[b + 1]])
        if mask is not None:
            bits = np.unpackbits(mask[b].cpu().numpy().view(np.uint8), bitorder="little")
            z[b, bits[:c["V"]] == 0] = -np.inf
    return {"logits": torch.from_numpy(z)}
