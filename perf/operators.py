"""Serving operators of the windowed paged cache: their plain forms, the calls
a user makes, and the cases they are timed on.

  decode         one new token per sequence attends to a sliding window of its
                 paged context and to its first tokens (sinks)
  decode_append  the same call, which also writes the new token's K and V
  prefill        a chunk of each sequence's last tokens, the same mask per row
  rope           rotary positions with several axes on q and k, and the write
                 of k and v into their cache slots

Token j is visible to the query at position p when j <= p and (p - j < window
or j < sinks).
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the smallest serving step: four short chats on a small model (launch latency)
        dict(name="decode_smallest", op="decode", seqs=4, q_heads=4, kv_heads=4, dim=64, type="f16",
             len_lo=1, len_hi=64, window=32, sinks=4, lens_seed=1),
        # one user deep in a long conversation: few rows, a long window
        dict(name="decode_one_user", op="decode", seqs=1, q_heads=32, kv_heads=8, dim=128, type="bf16",
             len_lo=32768, len_hi=32768, window=8192, sinks=4, lens_seed=2),
        # an ordinary batch of one-head-per-kv-head decoding, some contexts shorter than the window
        dict(name="decode_batch", op="decode", seqs=64, q_heads=32, kv_heads=32, dim=128, type="f16",
             len_lo=16, len_hi=2048, window=1024, sinks=4, lens_seed=3),
        # the largest: many long grouped-query contexts
        dict(name="decode_gqa_large", op="decode", seqs=128, q_heads=32, kv_heads=8, dim=128, type="bf16",
             len_lo=8192, len_hi=32768, window=4096, sinks=16, lens_seed=4),
        # odd sizes: ragged lengths with an empty one among them, 12 query heads on one kv head, a window that
        # starts inside a block
        dict(name="append_ragged", op="decode_append", seqs=37, q_heads=12, kv_heads=1, dim=64, type="f16",
             len_lo=0, len_hi=5000, window=777, sinks=5, lens_seed=5),
        # the decode step of a grouped-query model as a serving loop runs it
        dict(name="append_gqa", op="decode_append", seqs=48, q_heads=32, kv_heads=8, dim=128, type="bf16",
             len_lo=100, len_hi=8192, window=2048, sinks=4, lens_seed=6),
        # the tail of three prompts: few rows, odd lengths
        dict(name="prefill_small", op="prefill", seqs=3, q_heads=8, kv_heads=2, dim=64, type="f16", chunk_lo=1,
             chunk_hi=40, len_lo=40, len_hi=400, window=100, sinks=4, lens_seed=7),
        # one long prompt's next chunk while nothing else waits
        dict(name="prefill_one_chunk", op="prefill", seqs=1, q_heads=32, kv_heads=8, dim=128, type="bf16",
             chunk_lo=512, chunk_hi=512, len_lo=16384, len_hi=16384, window=4096, sinks=4, lens_seed=8),
        # a full step budget of chunks over long contexts
        dict(name="prefill_large", op="prefill", seqs=16, q_heads=32, kv_heads=8, dim=128, type="bf16",
             chunk_lo=512, chunk_hi=512, len_lo=512, len_hi=16384, window=4096, sinks=64, lens_seed=9),
        # one decode step's new tokens: launch latency
        dict(name="rope_decode", op="rope", tokens=64, q_heads=32, kv_heads=8, dim=128, type="bf16",
             sections="16 24 24", interleaved=False, theta=1000000.0),
        # plain one-axis positions on part of the head, neighbouring pairs, odd token count
        dict(name="rope_partial", op="rope", tokens=1023, q_heads=32, kv_heads=32, dim=128, type="f16",
             sections="32", interleaved=True, theta=10000.0),
        # a step budget of prompt tokens, text and video frames
        dict(name="rope_prefill", op="rope", tokens=8192, q_heads=32, kv_heads=8, dim=128, type="bf16",
             sections="16 24 24", interleaved=False, theta=1000000.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode_append", "prefill", "prefill", "rope"])
    dim = rng.choice([64, 128])
    kv = rng.choice([1, 2, 4, 8, 32])
    group = rng.choice([1, 1, 2, 4, 7, 8, 16]) if kv <= 8 else 1
    case = dict(op=op, q_heads=kv * group, kv_heads=kv, dim=dim, type=rng.choice(["f16", "bf16"]))
    if op == "rope":
        half = rng.choice([dim // 2, dim // 2, dim // 4, 16])
        axes = rng.choice([1, 2, 3, 4])
        cuts = sorted(rng.sample(range(1, half), axes - 1))
        case.update(tokens=_log(rng, 1, 8192), interleaved=rng.random() < 0.3,
                    sections=" ".join(str(b - a) for a, b in zip([0] + cuts, cuts + [half])),
                    theta=rng.choice([10000.0, 500000.0, 1000000.0]))
        return case
    window = _log(rng, 1, 8192)
    len_hi = _log(rng, 1, 32768)
    case.update(window=window, sinks=rng.choice([0, 1, 4, 5, 16, 64]), len_hi=len_hi,
                len_lo=rng.choice([0, 1, len_hi // 2, len_hi]), lens_seed=rng.randrange(1 << 30))
    case["len_lo"] = min(case["len_lo"], len_hi)
    if op == "prefill":
        case["chunk_hi"] = _log(rng, 1, 1024)
        case["chunk_lo"] = rng.choice([1, case["chunk_hi"]])
        # at most the largest case's score count: rows x visible tokens x heads
        budget = 8192 * 4160 * 32 * 128
        cost = case["chunk_hi"] * min(window + case["sinks"] + 1, len_hi) * kv * group * dim
        held = min(window + case["sinks"] + case["chunk_hi"], len_hi) * kv * dim
        case["seqs"] = min(_log(rng, 1, 32), max(1, budget // cost), max(1, 128 * 4112 * 8 * 128 // held))
        case["len_lo"] = max(1, case["len_lo"])
        return case
    budget = 128 * 4112 * 8 * 128  # at most the largest case's K bytes
    cost = min(window + case["sinks"], len_hi) * kv * dim
    case["seqs"] = min(_log(rng, 1, 256), max(1, budget // max(1, cost)))
    return case


def _sections(case):
    """Pairs of each axis."""
    return [int(x) for x in case["sections"].split()]


def _lens(case):
    """(context lengths, chunk lengths): fixed by the case, whatever the seed."""
    rng = np.random.default_rng(case["lens_seed"])
    lens = rng.integers(case["len_lo"], case["len_hi"] + 1, size=case["seqs"])
    if case["op"] != "prefill":
        return lens, None
    chunk = np.minimum(rng.integers(case["chunk_lo"], case["chunk_hi"] + 1, size=case["seqs"]), lens)
    return lens, chunk


def _visible(case, first, last):
    """Tokens visible to any query at positions first .. last."""
    lo = max(0, first - case["window"] + 1)
    return last + 1 - lo + min(case["sinks"], lo)


def work(case):
    Hq, H, d = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "rope":
        T, axes, half = case["tokens"], len(_sections(case)), sum(_sections(case))
        return {"bytes": 2 * T * (Hq + 2 * H) * d * 2 + T * (4 * axes + 8) + 4 * half,
                "flops": 6 * T * (Hq + H) * half}
    lens, chunk = _lens(case)
    nbytes = flops = 0
    for s in range(case["seqs"]):
        L = int(lens[s])
        n = 1 if chunk is None else int(chunk[s])
        if chunk is None:
            nbytes += 2 * Hq * d * 2  # q and out, an empty row's too
        else:
            nbytes += 2 * n * Hq * d * 2
        nbytes += 4
        if L == 0 or n == 0:
            continue
        seen = _visible(case, L - n, L - 1)
        nbytes += seen * H * d * 2 * 2 + 4 * -(-seen // BLOCK)
        if case["op"] == "decode_append":
            nbytes += 2 * H * d * 2 * 2
        pos = np.arange(L - n, L)
        lo = np.maximum(0, pos - case["window"] + 1)
        flops += 4 * Hq * d * int((pos + 1 - lo + np.minimum(case["sinks"], lo)).sum())
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------------ inputs
def _rope_inputs(case, gen, dtype):
    T, Hq, H, d = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
    qkv = torch.randn(T, (Hq + 2 * H) * d, generator=gen, device="cuda").to(dtype)
    axes, half = len(_sections(case)), sum(_sections(case))
    # text advances every axis together; frames of a video hold the time and walk over rows and columns; the
    # chunk starts anywhere in a long context
    start = torch.randint(0, 100000, (1,), generator=gen, device="cuda")
    t = torch.arange(T, device="cuda")
    frame = (t // 256) % 2 == 1
    pos = torch.empty(axes, T, dtype=torch.int32, device="cuda")
    for a in range(axes):
        inside = t // 256 if a == 0 else (t % 256) // 16 if a == 1 else t % 16
        pos[a] = (start + torch.where(frame, t // 256 * 256 + inside, t)).to(torch.int32)
    slots_pool = -(-T // BLOCK) + 8  # blocks
    slots = torch.randperm(slots_pool * BLOCK, generator=gen, device="cuda")[:T]
    if T > 8:
        slots[T // 2] = -1  # a padded token
    kc = torch.randn(slots_pool, H, BLOCK, d, generator=gen, device="cuda").to(dtype)
    vc = torch.randn(slots_pool, H, BLOCK, d, generator=gen, device="cuda").to(dtype)
    inv_freq = (float(case["theta"]) ** (-np.arange(half) / half)).astype(np.float32)
    axis = np.repeat(np.arange(axes), _sections(case)).astype(np.int32)
    return dict(case=case, qkv=qkv, positions=pos, slots=slots, kc=kc, vc=vc, inv_freq=inv_freq, axis=axis)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 17)
    dtype = TYPES[case["type"]]
    Hq, H, d = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "rope":
        st = _rope_inputs(case, gen, dtype)
        if own:
            import paged_kv_cache_425_b200 as pk
            st["rope"] = pk.Rope(st["inv_freq"], st["axis"], interleaved=case["interleaved"])
            st["q_out"] = torch.empty(case["tokens"], Hq, d, dtype=dtype, device="cuda")
        return st
    lens, chunk = _lens(case)
    S = case["seqs"]
    # the tables of a cache that freed the pages behind the window: only visible blocks are held
    maxb = max(1, -(-int(lens.max()) // BLOCK))
    held = np.zeros((S, maxb), bool)
    for s in range(S):
        L = int(lens[s])
        n = 1 if chunk is None else int(chunk[s])
        lo = max(0, L - n - case["window"] + 1)
        nblk = -(-L // BLOCK)
        held[s, lo // BLOCK:nblk] = True
        held[s, :min(nblk, -(-case["sinks"] // BLOCK))] = True
    blocks = int(held.sum())
    pool = blocks + max(2, blocks // 10)
    ids = torch.randperm(pool, generator=gen, device="cuda")[:blocks].to(torch.int32)
    tables = torch.full((S, maxb), -1, dtype=torch.int32, device="cuda")
    tables[torch.from_numpy(held).cuda()] = ids
    kc = torch.empty(pool, H, BLOCK, d, dtype=dtype, device="cuda")
    vc = torch.empty(pool, H, BLOCK, d, dtype=dtype, device="cuda")
    kc.normal_(generator=gen)
    vc.normal_(generator=gen)
    rows = S if chunk is None else int(chunk.sum())
    q = torch.randn(rows, Hq, d, generator=gen, device="cuda").to(dtype)
    st = dict(case=case, q=q, kc=kc, vc=vc, tables=tables, host_lens=[int(x) for x in lens],
              lens=torch.from_numpy(lens.astype(np.int32)).cuda(), scale=1.0 / math.sqrt(d))
    if case["op"] == "decode_append":
        st["k_new"] = torch.randn(S, H, d, generator=gen, device="cuda").to(dtype)
        st["v_new"] = torch.randn(S, H, d, generator=gen, device="cuda").to(dtype)
    if chunk is not None:
        start = np.concatenate([[0], np.cumsum(chunk)])
        st["host_start"] = [int(x) for x in start]
        st["start"] = torch.from_numpy(start.astype(np.int32)).cuda()
        st["max_chunk"] = int(chunk.max())
    if own:
        import paged_kv_cache_425_b200 as pk
        st["out"] = torch.empty_like(q)
        if chunk is None:
            n = pk.decode_window_workspace_size(S, Hq, H, d, maxb, case["window"], case["sinks"])
        else:
            n = pk.prefill_window_workspace_size(S, rows, st["max_chunk"], Hq, H, d, maxb, case["window"],
                                                 case["sinks"])
        st["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    return st


# ------------------------------------------------------------------ the calls
def run(state):
    return _call(state) if own else _plain(state)


def _split_qkv(state):
    case = state["case"]
    Hq, H, d = case["q_heads"], case["kv_heads"], case["dim"]
    T = case["tokens"]
    q, k, v = state["qkv"].split([Hq * d, H * d, H * d], dim=1)
    return q.view(T, Hq, d), k.view(T, H, d), v.view(T, H, d)


def _call(state):
    import paged_kv_cache_425_b200 as pk
    case = state["case"]
    op = case["op"]
    if op == "rope":
        q, k, v = _split_qkv(state)
        pk.rope_and_cache(state["q_out"], q, k, v, state["kc"], state["vc"], state["slots"], state["positions"],
                          state["rope"])
        return state["q_out"], state["kc"], state["vc"]
    if op == "decode":
        pk.decode_window(state["out"], state["q"], state["kc"], state["vc"], state["tables"], state["lens"],
                         case["kv_heads"], state["scale"], case["window"], case["sinks"],
                         workspace=state["workspace"])
        return state["out"]
    if op == "decode_append":
        pk.decode_append_window(state["out"], state["q"], state["k_new"], state["v_new"], state["kc"], state["vc"],
                                state["tables"], state["lens"], case["kv_heads"], state["scale"], case["window"],
                                case["sinks"], workspace=state["workspace"])
        return state["out"], state["kc"], state["vc"]
    pk.prefill_window(state["out"], state["q"], state["kc"], state["vc"], state["tables"], state["lens"],
                      state["start"], state["max_chunk"], case["kv_heads"], state["scale"], case["window"],
                      case["sinks"], workspace=state["workspace"])
    return state["out"]


# ------------------------------------------------------------------ plain forms
def _plain(state):
    op = state["case"]["op"]
    if op == "rope":
        return _plain_rope(state)
    if op == "prefill":
        return _plain_prefill(state)
    if op == "decode":
        return _plain_decode(state, state["kc"], state["vc"])
    kc, vc = state["kc"], state["vc"]
    last = (state["lens"].long() - 1).clamp(min=0)
    block = state["tables"].long().gather(1, (last // BLOCK)[:, None])[:, 0]
    live = state["lens"] > 0
    block, off = block[live], (last % BLOCK)[live]
    kc[block, :, off] = state["k_new"][live]
    vc[block, :, off] = state["v_new"][live]
    return _plain_decode(state, kc, vc), kc, vc


def _plain_decode(state, kc, vc):
    case = state["case"]
    H, d, S = case["kv_heads"], case["dim"], case["seqs"]
    q, lens, tables = state["q"], state["lens"].long(), state["tables"].long()
    span = min(case["window"], max(max(state["host_lens"]), 1))
    lo = (lens - case["window"]).clamp(min=0)
    pos = lo[:, None] + torch.arange(span, device=q.device)
    ok = pos < lens[:, None]
    if case["sinks"]:
        first = torch.arange(min(case["sinks"], max(max(state["host_lens"]), 1)), device=q.device).expand(S, -1)
        pos = torch.cat([first, pos], 1)
        ok = torch.cat([first < lo[:, None], ok], 1)
    block = tables.gather(1, torch.where(ok, pos // BLOCK, 0)).clamp(min=0)
    off = pos % BLOCK
    K = kc[block, :, off].float().transpose(1, 2)  # S, H, n, d
    V = vc[block, :, off].float().transpose(1, 2)
    Q = q.float().view(S, H, -1, d)
    x = (Q @ K.transpose(2, 3)) * state["scale"]
    x = torch.where(ok[:, None, None, :], x, -torch.inf)
    m = x.amax(3, keepdim=True)
    p = torch.exp(x - torch.where(m == -torch.inf, 0.0, m))
    den = p.sum(3, keepdim=True)
    o = (p @ V) / torch.where(den == 0, 1.0, den)
    return o.view(S, -1, d).to(q.dtype)


def _plain_prefill(state):
    case = state["case"]
    H, d = case["kv_heads"], case["dim"]
    q = state["q"]
    out = torch.empty_like(q)
    for s, L in enumerate(state["host_lens"]):
        r0, r1 = state["host_start"][s], state["host_start"][s + 1]
        for a in range(r0, r1, 512):
            b = min(r1, a + 512)
            first, last = L - (r1 - a), L - (r1 - b) - 1
            lo = max(0, first - case["window"] + 1)
            ns = min(case["sinks"], lo)
            keys = torch.cat([torch.arange(ns, device=q.device), torch.arange(lo, last + 1, device=q.device)])
            block = state["tables"][s].long()[keys // BLOCK]
            K = state["kc"][block, :, keys % BLOCK].float().transpose(0, 1)  # H, n, d
            V = state["vc"][block, :, keys % BLOCK].float().transpose(0, 1)
            Q = q[a:b].float().view(b - a, H, -1, d).permute(1, 2, 0, 3)  # H, G, rows, d
            p = torch.arange(first, last + 1, device=q.device)[:, None]
            see = (keys <= p) & ((p - keys < case["window"]) | (keys < case["sinks"]))
            x = torch.where(see, (Q @ K[:, None].transpose(2, 3)) * state["scale"], -torch.inf)
            w = torch.exp(x - x.amax(3, keepdim=True))
            o = (w @ V[:, None]) / w.sum(3, keepdim=True)
            out[a:b] = o.permute(2, 0, 1, 3).reshape(b - a, -1, d).to(q.dtype)
    return out


def _plain_rope(state):
    case = state["case"]
    q, k, v = _split_qkv(state)
    dev = q.device
    half = sum(_sections(case))
    pos = state["positions"].double()[torch.from_numpy(state["axis"]).to(dev).long()]  # half, T
    angle = pos.T * torch.from_numpy(state["inv_freq"]).to(dev).double()
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def rotate(x):
        y = x.float()
        if case["interleaved"]:
            a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
            turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(2)
        else:
            a, b = y[..., :half], y[..., half:2 * half]
            turned = torch.cat([a * c - b * s, b * c + a * s], -1)
        return torch.cat([turned, y[..., 2 * half:]], -1).to(x.dtype)

    kept = (state["slots"] >= 0).nonzero()[:, 0]
    block, off = state["slots"][kept] // BLOCK, state["slots"][kept] % BLOCK
    state["kc"][block, :, off] = rotate(k)[kept]
    state["vc"][block, :, off] = v[kept]
    return rotate(q), state["kc"], state["vc"]


# ------------------------------------------------------------------ 64 bits, from the definition
def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return _exact_rope(state)
    if op == "prefill":
        start = state["host_start"]
    else:
        start = list(range(case["seqs"] + 1))
    if op == "decode_append":
        for s, L in enumerate(state["host_lens"]):
            if L > 0:
                b = int(state["tables"][s, (L - 1) // BLOCK])
                state["kc"][b, :, (L - 1) % BLOCK] = state["k_new"][s]
                state["vc"][b, :, (L - 1) % BLOCK] = state["v_new"][s]
    q = state["q"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    G = case["q_heads"] // case["kv_heads"]
    for s, L in enumerate(state["host_lens"]):
        rows = start[s + 1] - start[s]
        if L == 0 or rows == 0:
            continue
        first = L - rows
        floor = max(0, first + 1 - case["window"]) // BLOCK  # first block inside any row's window
        head = min(floor, -(-case["sinks"] // BLOCK))
        blocks = list(range(head)) + list(range(floor, -(-L // BLOCK)))
        index = torch.tensor(blocks, device=q.device)
        j = (index[:, None] * BLOCK + torch.arange(BLOCK, device=q.device)).flatten()
        keep = j < L
        ids = state["tables"][s, index].long()
        for h in range(case["kv_heads"]):
            K = state["kc"][ids, h].double().flatten(0, 1)[keep]
            V = state["vc"][ids, h].double().flatten(0, 1)[keep]
            jj = j[keep]
            for a in range(0, rows, 256):
                b = min(rows, a + 256)
                Q = q[start[s] + a:start[s] + b, h * G:(h + 1) * G].double()
                p = first + torch.arange(a, b, device=q.device)
                hidden = (jj[None] > p[:, None]) | ((jj[None] <= p[:, None] - case["window"]) &
                                                   (jj[None] >= case["sinks"]))
                x = torch.einsum("rgd,nd->rgn", Q, K) * state["scale"]
                w = torch.softmax(x.masked_fill(hidden[:, None], -math.inf), -1)
                out[start[s] + a:start[s] + b, h * G:(h + 1) * G] = torch.einsum("rgn,nd->rgd", w, V)
    if op == "decode_append":
        return out, state["kc"].double(), state["vc"].double()
    return out


def _exact_rope(state):
    case = state["case"]
    Hq, H, d, T = case["q_heads"], case["kv_heads"], case["dim"], case["tokens"]
    x = state["qkv"].double().view(T, Hq + 2 * H, d)
    half = sum(_sections(case))
    if case["interleaved"]:
        even = torch.arange(0, 2 * half, 2, device=x.device)
        odd = even + 1
    else:
        even = torch.arange(half, device=x.device)
        odd = even + half
    turn = torch.empty(T, half, dtype=torch.float64, device=x.device)
    for i in range(half):
        turn[:, i] = state["positions"][int(state["axis"][i])].double() * float(state["inv_freq"][i])
    z = torch.polar(torch.ones_like(turn), turn)[:, None]
    y = x.clone()
    qk = torch.complex(x[:, :Hq + H, even], x[:, :Hq + H, odd]) * z
    y[:, :Hq + H, even], y[:, :Hq + H, odd] = qk.real, qk.imag
    kc, vc = state["kc"].double(), state["vc"].double()
    slots = state["slots"].tolist()
    rows = [t for t in range(T) if slots[t] >= 0]
    where = torch.tensor([slots[t] for t in rows], device=x.device)
    kc.transpose(1, 2)[where // BLOCK, where % BLOCK] = y[rows, Hq:Hq + H]
    vc.transpose(1, 2)[where // BLOCK, where % BLOCK] = y[rows, Hq + H:]
    return y[:, :Hq], kc, vc
