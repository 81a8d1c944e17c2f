"""Cases of the paged KV cache: rotary positions, new rows rotated and written into pages, attention of trees and
chunks over pages, moving an accepted path.

A page holds `page` slots of every KV head: k_pages, v_pages [pages][Hkv][page][D]; row b of the block table names
request b's pages in the order of its slots.  Request b's new rows (a tree's nodes or a chunk's tokens) take the slots
from its prefix length on.  A row's position is its request's start plus its depth in the tree, or its place in the
chunk.
"""
import math

import numpy as np
import torch

own = False

MAX_NODES = 128


def dtype_of(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


# ------------------------------------------------------------------ shapes
def counts(case):
    """New rows and prefix of each request: a batch's requests shrink from the first on by up to `spread`."""
    B = case["B"]
    n = [max(1, case["N"] - int(case["spread"] * case["N"] * b / B)) for b in range(B)]
    L = [max(0, case["L"] - int(case["spread"] * case["L"] * b / B)) for b in range(B)]
    return n, L


def listed():
    rot = dict(rot=128, layout="half", base=500000.0, scaling="bands", factor=8.0)
    gqa = dict(Hq=64, Hkv=8, D=128)
    attn = dict(op="attn", dtype="bf16", D=128, spread=0.0, shape="tree")
    return [
        # plain decoding of four requests behind 8192 tokens: queries and keys of the fused projection
        dict(rot, **gqa, name="rope_tokens", op="rope", dtype="bf16", B=4, N=1, L=8192, spread=0.0, shape="chunk", fused=True),
        # prompts of eight requests, half of each head rotated, interleaved pairs, a context stretched 16 times
        dict(name="rope_prompts", op="rope", dtype="bf16", B=8, Hq=32, Hkv=8, D=128, N=8192, L=0, spread=0.5, shape="chunk",
             fused=False, rot=64, layout="interleaved", base=10000.0, scaling="yarn", factor=16.0),
        # one step's tree of a model of 32 heads goes into its pages
        dict(name="write_step_tree", op="write", dtype="bf16", B=1, Hq=32, Hkv=32, D=128, N=64, L=2048, spread=0.0,
             shape="tree", fused=False, page=16, rot=128, layout="half", base=10000.0, scaling="none", factor=1.0),
        # chunks of eight prompts, rows taken from the fused projection
        dict(rot, **gqa, name="write_chunks", op="write", dtype="bf16", B=8, N=2048, L=4096, spread=0.3, shape="chunk",
             fused=True, page=64),
        # the smallest step: an 8-node tree behind 128 tokens, fp32
        dict(attn, name="attn_tiny_fp32", dtype="fp32", B=1, Hq=4, Hkv=4, D=64, N=8, L=128, page=16),
        # plain decoding: one new token per request, 8 query heads per KV head
        dict(attn, name="attn_single_token", B=4, Hq=64, Hkv=8, N=1, L=8192, page=64, shape="chain"),
        # one request's 64-node tree, 32 heads
        dict(attn, name="attn_tree_64", B=1, Hq=32, Hkv=32, N=64, L=2048, page=16),
        # 128-node trees of four requests, 8 query heads per KV head
        dict(attn, name="attn_tree_128_gqa", B=4, Hq=64, Hkv=8, N=128, L=8192, page=64),
        # a chain of 6 drafted tokens behind long prefixes of different lengths
        dict(attn, name="attn_long_chain", B=8, Hq=32, Hkv=32, N=6, L=32768, spread=0.2, page=128, shape="chain"),
        # a chunk of 2048 prompt tokens behind the 16384 already in the cache
        dict(attn, name="attn_chunk", B=1, Hq=64, Hkv=8, N=2048, L=16384, page=64, shape="chunk"),
        # the accepted path of one tree moves behind its prefix
        dict(name="compact_tree", op="compact", dtype="bf16", B=1, Hkv=32, D=128, N=64, L=2048, spread=0.0, page=16,
             shape="tree"),
        # the same for a batch of sixteen ragged trees
        dict(name="compact_batch", op="compact", dtype="bf16", B=16, Hkv=32, D=128, N=96, L=1024, spread=0.8, page=64,
             shape="tree"),
    ]


def between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "attn", "rope", "write", "write", "compact"])
    case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "bf16", "fp32"]), D=rng.choice([64, 128, 128]),
                B=between(rng, 1, 16), Hkv=rng.choice([1, 2, 4, 8, 32]), page=rng.choice([16, 16, 32, 64, 128, 256]),
                spread=rng.choice([0.0, round(rng.uniform(0.05, 0.95), 2)]), L=between(rng, 1, 32768) - 1)
    G, D = rng.choice([1, 1, 2, 3, 4, 5, 8, 8]), case["D"]
    case["Hq"] = case["Hkv"] * G
    case["shape"] = rng.choice(["tree", "tree", "chain", "chunk"])
    top = 4096 if case["shape"] == "chunk" else MAX_NODES
    case["N"] = between(rng, 1, top)
    if op == "compact":
        case.update(shape="tree", N=between(rng, 1, MAX_NODES), L=min(case["L"], 2048), dtype="bf16")
        return case
    if op in ("rope", "write"):
        case.update(fused=rng.random() < 0.5, layout=rng.choice(["half", "interleaved"]),
                    rot=rng.choice([D, D, D // 2, D // 4, 24]), base=rng.choice([10000.0, 500000.0]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn", "bands"]),
                    factor=rng.choice([2.0, 8.0, 16.0]), L=min(case["L"], 8192))
        heads = case["Hq"] + 2 * case["Hkv"]
        while case["B"] * case["N"] * heads * D * (2 if case["dtype"] == "fp32" else 1) > 16384 * 80 * 128:
            case["B"], case["N"] = max(1, case["B"] // 2), max(1, case["N"] // 2 + case["N"] % 2)
        return case
    if case["dtype"] == "fp32":
        case["L"], case["N"] = min(case["L"], 4096), min(case["N"], 512)
    size = 8 if case["dtype"] == "fp32" else 1     # fp32 has no tensor cores of its own precision
    while case["B"] > 1 and (case["B"] * case["Hkv"] * (case["L"] + case["N"]) > 8 * 32 * 30000
                             or size * case["B"] * case["Hq"] * case["N"] * (case["L"] + case["N"]) > 64 * 2048 * 17408):
        case["B"] //= 2
    while size * case["B"] * case["Hq"] * case["N"] * (case["L"] + case["N"]) > 64 * 2048 * 17408:
        case["L"] //= 2
        case["N"] -= case["N"] // 4
    return case


# ------------------------------------------------------------------ inputs
def parents_of(case, nb, rs):
    return [-1] + [i - 1 if case["shape"] != "tree" else int(rs.randint(max(0, i - 12), i)) for i in range(1, nb)]


def trees(case, rs):
    """Ancestor masks (128 bits a node, as four words), depths and an accepted path of every request."""
    words, depths, paths = [], [], []
    for nb in counts(case)[0]:
        sets, depth = [], []
        for i, p in enumerate(parents_of(case, nb, rs)):
            sets.append((sets[p] if p >= 0 else 0) | 1 << i)
            depth.append(depth[p] + 1 if p >= 0 else 0)
        words += [[s >> 32 * w & 0xFFFFFFFF for w in range(4)] for s in sets]
        depths += depth
        last = sets[int(rs.randint(0, nb))]
        paths.append([i for i in range(nb) if last >> i & 1])
    return words, depths, paths


def pages(case, rs):
    """A block table over pages in no order, as a pool that has served many requests hands them out; -1 behind a
    request's last page."""
    n, L = counts(case)
    need = [-(-(a + b) // case["page"]) for a, b in zip(n, L)]
    total = sum(need) + 3
    order = rs.permutation(total)
    table = np.full((case["B"], max(need)), -1, dtype=np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    return table, total


def pool(case, total, gen):
    """Keys and values as attention finds them; anything at all, NaN here, where no request has written."""
    shape = (total, case["Hkv"], case["page"], case["D"])
    return [torch.randn(shape, device="cuda", generator=gen, dtype=dtype_of(case)) for _ in range(2)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rs = np.random.RandomState(seed % (1 << 31))
    n, L = counts(case)
    off = np.concatenate([[0], np.cumsum(n)])
    T, dt, D, op = int(off[-1]), dtype_of(case), case["D"], case["op"]
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    st = dict(case=case, off=i32(off), lens=i32(L), status=torch.zeros(case["B"], dtype=torch.int32, device="cuda"), T=T)
    st["depth"] = None
    if case["shape"] != "chunk":
        words, depth, paths = trees(case, rs)
        st["depth"] = i32(depth)
    if op in ("rope", "write"):
        Hq, Hkv = case["Hq"], case["Hkv"]
        heads = Hq + 2 * Hkv
        size = torch.exp(0.6 * torch.randn((heads, D), device="cuda", generator=gen))
        x = (torch.randn((T, heads, D), device="cuda", generator=gen) * size).to(dt)
        parts = [x[:, :Hq + Hkv]] if op == "rope" else [x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]]
        st["rows"] = parts if case["fused"] else [p.contiguous() for p in parts]
        if own:
            import token_tree_verification_gb300 as ttv
            st["rope"] = ttv.rope_table(case["rot"], case["base"], case["scaling"], case["factor"], original=4096)
    if op == "rope":
        return st
    table, total = pages(case, rs)
    st["table"] = i32(table)
    if op == "write":
        st["pages"] = [torch.zeros((total, case["Hkv"], case["page"], D), dtype=dt, device="cuda") for _ in range(2)]
        return st
    st["pages"] = pool(case, total, gen)
    if op == "compact":
        W = max(len(p) for p in paths)
        st.update(path=i32([p + [-1] * (W - len(p)) for p in paths]), accept=i32([len(p) - 1 for p in paths]))
        return st
    written = torch.zeros((total, case["page"]), dtype=torch.bool, device="cuda")
    for b in range(case["B"]):
        slot = torch.arange(L[b] + n[b], device="cuda")
        written[st["table"][b].long()[slot // case["page"]], slot % case["page"]] = True
    dead = torch.nonzero(~written)
    for x in st["pages"]:
        x[dead[:, 0], :, dead[:, 1]] = math.nan
    st["mask"] = None
    if case["shape"] != "chunk":
        st["mask"] = torch.tensor(np.array(words, dtype=np.uint32).view(np.int32), device="cuda")
    st["q"] = (2.0 * torch.randn((T, case["Hq"], D), device="cuda", generator=gen)).to(dt)
    st["max_prefix"] = max(L)
    return st


# ------------------------------------------------------------------ plain forms
def frequencies(case):
    """Radians a position of each rotated pair, and the factor of cosine and sine."""
    r, base, f, original = case["rot"], case["base"], case["factor"], 4096
    kind, scale = case["scaling"], 1.0
    if kind == "ntk":
        base *= f ** (r / (r - 2))
    theta = [base ** (-2 * i / r) for i in range(r // 2)]
    if kind == "linear":
        theta = [t / f for t in theta]
    if kind == "yarn":
        turns = lambda b: r * math.log(original / (2 * math.pi * b)) / (2 * math.log(base))  # noqa: E731
        low, high = max(0, math.floor(turns(32.0))), min(r - 1, math.ceil(turns(1.0)))
        ramp = [min(1.0, max(0.0, (i - low) / max(high - low, 0.001))) for i in range(r // 2)]
        theta = [t / f * g + t * (1 - g) for t, g in zip(theta, ramp)]
        scale = 0.1 * math.log(f) + 1
    if kind == "bands":
        mix = [min(1.0, max(0.0, (original * t / (2 * math.pi) - 1.0) / (4.0 - 1.0))) for t in theta]
        theta = [(1 - m) * t / f + m * t for t, m in zip(theta, mix)]
    return theta, scale


def requests_of(st):
    """Request and place in it of every packed row."""
    row = torch.arange(st["T"], device="cuda")
    b = torch.searchsorted(st["off"][1:].long().contiguous(), row, right=True)
    return b, row - st["off"].long()[b]


def plain_rotate(st, x):
    case, r = st["case"], st["case"]["rot"]
    b, place = requests_of(st)
    position = st["lens"].long()[b] + (place if st["depth"] is None else st["depth"].long())
    theta, scale = frequencies(case)
    angle = position.double()[:, None] * torch.tensor(theta, dtype=torch.float64, device="cuda")
    cos, sin = (torch.cos(angle) * scale).float()[:, None], (torch.sin(angle) * scale).float()[:, None]
    x = x.float()
    if case["layout"] == "half":
        p, q = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([p * cos - q * sin, p * sin + q * cos], -1)
    else:
        p, q = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([p * cos - q * sin, p * sin + q * cos], -1).flatten(-2)
    return torch.cat([turned, x[..., r:]], -1).to(dtype_of(case))


def plain_write(st):
    q, k, v = st["rows"]
    b, place = requests_of(st)
    slot = st["lens"].long()[b] + place
    page, at = st["table"].long()[b, slot // st["case"]["page"]], slot % st["case"]["page"]
    st["pages"][0][page, :, at] = plain_rotate(st, k)
    st["pages"][1][page, :, at] = v
    return plain_rotate(st, q), st["pages"][0], st["pages"][1]


def plain_compact(st):
    P, L, path, acc = st["case"]["page"], st["lens"].long(), st["path"].long(), st["accept"].long()
    step = torch.arange(path.shape[1], device="cuda")
    b, j = torch.nonzero((step[None, :] >= 1) & (step[None, :] <= acc[:, None]), as_tuple=True)
    old, new = L[b] + path[b, j], L[b] + j
    table = st["table"].long()
    for x in st["pages"]:
        rows = x[table[b, old // P], :, old % P]
        x[table[b, new // P], :, new % P] = rows
    return st["lens"] + 1 + st["accept"], st["pages"][0], st["pages"][1]


def plain_attn(st):
    case, q = st["case"], st["q"]
    Hkv, G, D, P = case["Hkv"], case["Hq"] // case["Hkv"], case["D"], case["page"]
    out, at = torch.empty_like(q), 0
    for b, (n, L) in enumerate(zip(*counts(case))):
        keys = L + n
        used = st["table"][b, :-(-keys // P)].long()
        k, v = (x[used].transpose(0, 1).flatten(1, 2)[:, :keys].float() for x in st["pages"])      # [Hkv][keys][D]
        rows = q[at:at + n].float().unflatten(1, (Hkv, G))                                         # [n][Hkv][G][D]
        slot = torch.arange(keys, device="cuda")
        step = max(1, 2 ** 28 // (Hkv * G * keys))
        for i in range(0, n, step):
            m = min(step, n - i)
            if st["mask"] is None:
                ok = slot[None, :] <= L + i + torch.arange(m, device="cuda")[:, None]
            else:
                bit = torch.clamp(slot - L, 0, MAX_NODES - 1)
                word = st["mask"][at + i:at + i + m][:, bit // 32]
                ok = (word >> (bit % 32).int() & 1).bool() | (slot < L)
            x = rows[i:i + m].permute(1, 0, 2, 3).reshape(Hkv, m * G, D)
            score = torch.matmul(x, k.transpose(1, 2)) / math.sqrt(D)
            score = score.unflatten(1, (m, G)).masked_fill_(~ok[None, :, None, :], -math.inf)
            p = torch.exp(score - score.amax(-1, keepdim=True))
            o = torch.matmul(p.flatten(1, 2), v).unflatten(1, (m, G)) / p.sum(-1, keepdim=True)
            out[at + i:at + i + m] = o.permute(1, 0, 2, 3).flatten(1, 2).to(q.dtype)
        at += n
    return out


def run(state):
    if own:
        return run_own(state)
    op = state["case"]["op"]
    if op == "rope":
        return plain_rotate(state, state["rows"][0])
    return {"write": plain_write, "compact": plain_compact, "attn": plain_attn}[op](state)


def run_own(st):
    import token_tree_verification_gb300 as ttv
    case = st["case"]
    if case["op"] == "rope":
        return ttv.rope(st["rows"][0], st["rope"], st["lens"], st["off"], st["status"], depth=st["depth"],
                        interleaved=case["layout"] == "interleaved")
    kp, vp = st["pages"]
    if case["op"] == "write":
        q, k, v = st["rows"]
        return ttv.rope_write_paged(q, k, v, kp, vp, st["table"], st["lens"], st["off"], st["status"], st["rope"],
                                    depth=st["depth"], interleaved=case["layout"] == "interleaved"), kp, vp
    if case["op"] == "compact":
        return ttv.kv_compact_paged(kp, vp, st["table"], st["lens"], st["off"], st["path"], st["accept"],
                                    st["status"]), kp, vp
    return ttv.tree_attn_paged(st["q"], kp, vp, st["table"], st["lens"], st["off"], st["mask"], st["max_prefix"],
                               st["status"], causal=st["mask"] is None)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    n, L = counts(case)
    T, D, e = sum(n), case["D"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("rope", "write"):
        turned = case["Hq"] + case["Hkv"]
        heads = turned + (case["Hkv"] if case["op"] == "write" else 0)
        return {"bytes": 2 * T * heads * D * e, "flops": 3 * T * turned * case["rot"]}
    if case["op"] == "compact":      # a path's rows, read and written; its length is the tree's depth
        moved = sum(int(math.log2(a + 1)) for a in n)
        return {"bytes": 2 * 2 * moved * case["Hkv"] * D * e, "flops": 0}
    seen = sum(a * b + (a * (a + 1) // 2 if case["shape"] != "tree" else a) for a, b in zip(n, L))
    bytes_ = sum(a + b for a, b in zip(n, L)) * case["Hkv"] * 2 * D * e + 2 * T * case["Hq"] * D * e
    return {"bytes": bytes_, "flops": 4 * D * case["Hq"] * seen}


# ------------------------------------------------------------------ from the definitions, in 64 bits
def turn(x, case, positions):
    """Rows as complex numbers times exp(i position theta)."""
    r, x = case["rot"], x.double()
    i = torch.arange(r // 2, dtype=torch.float64, device="cuda")
    base, f, scale = case["base"], case["factor"], 1.0
    if case["scaling"] == "ntk":
        base = math.exp(math.log(base) + r / (r - 2) * math.log(f))
    theta = torch.exp(-2 * i / r * math.log(base))
    if case["scaling"] == "linear":
        theta = theta / f
    elif case["scaling"] == "yarn":
        pair = [r / 2 * math.log(4096 / (2 * math.pi * b)) / math.log(base) for b in (32.0, 1.0)]
        first, last = max(0, math.floor(pair[0])), min(r - 1, math.ceil(pair[1]))
        slow = torch.clamp((i - first) / max(last - first, 0.001), 0, 1)
        theta = theta * (1 - slow + slow / f)
        scale = 1 + math.log(f) / 10
    elif case["scaling"] == "bands":
        length = 2 * math.pi / theta
        keep = torch.clamp((4096 / length - 1) / 3, 0, 1)
        theta = theta * (keep + (1 - keep) / f)
    a, b = (x[..., :r // 2], x[..., r // 2:r]) if case["layout"] == "half" else (x[..., 0:r:2], x[..., 1:r:2])
    angle = torch.tensor(positions, dtype=torch.float64, device="cuda")[:, None, None] * theta
    z = torch.complex(a, b) * torch.polar(torch.full_like(angle, scale), angle)
    y = x.clone()
    if case["layout"] == "half":
        y[..., :r // 2], y[..., r // 2:r] = z.real, z.imag
    else:
        y[..., 0:r:2], y[..., 1:r:2] = z.real, z.imag
    return y


def exact(case, seed):
    st = prepare(case, seed)
    n, L = counts(case)
    off = [0] + list(np.cumsum(n))
    depth = None if st["depth"] is None else st["depth"].tolist()
    if case["op"] in ("rope", "write"):
        positions = [L[b] + (t - off[b] if depth is None else depth[t]) for b in range(case["B"])
                     for t in range(off[b], off[b + 1])]
    if case["op"] == "rope":
        return turn(st["rows"][0], case, positions)
    P, table = case["page"], st["table"].tolist()
    place = lambda b, s: (table[b][s // P], s % P)  # noqa: E731
    if case["op"] == "write":
        kp, vp = (x.double() for x in st["pages"])
        at = [place(b, L[b] + t - off[b]) for b in range(case["B"]) for t in range(off[b], off[b + 1])]
        pg, sl = (torch.tensor([p[i] for p in at], device="cuda") for i in range(2))
        kp[pg, :, sl], vp[pg, :, sl] = turn(st["rows"][1], case, positions), st["rows"][2].double()
        return turn(st["rows"][0], case, positions), kp, vp
    if case["op"] == "compact":
        lens, new = [], [x.clone() for x in st["pages"]]
        for b in range(case["B"]):
            acc = int(st["accept"][b])
            for j, node in enumerate(st["path"][b, 1:acc + 1].tolist(), 1):
                (p0, s0), (p1, s1) = place(b, L[b] + node), place(b, L[b] + j)
                for x, y in zip(st["pages"], new):
                    y[p1, :, s1] = x[p0, :, s0]
            lens.append(L[b] + 1 + acc)
        return torch.tensor(lens, dtype=torch.int32), new[0].double(), new[1].double()
    D, H, G = case["D"], case["Hkv"], case["Hq"] // case["Hkv"]
    if 4 * D * H * G * sum(a * (a + b) for a, b in zip(n, L)) > 4e12:
        return None
    out = torch.empty((off[-1], H * G, D), dtype=torch.float64, device="cuda")
    words = None if st["mask"] is None else st["mask"].cpu().numpy().view(np.uint32)
    for b in range(case["B"]):
        keys = L[b] + n[b]
        see = torch.ones((n[b], keys), dtype=torch.bool, device="cuda")
        if words is None:
            see = see.tril(L[b])
        else:
            tree = [[bool(words[off[b] + i][a // 32] >> np.uint32(a % 32) & 1) for a in range(n[b])] for i in range(n[b])]
            see[:, L[b]:] = torch.tensor(tree, device="cuda")
        used = torch.tensor(table[b][:-(-keys // P)], device="cuda")
        for h in range(H):
            k, v = (x[used, h].reshape(-1, D)[:keys].double() for x in st["pages"])
            for i in range(0, n[b], 512):
                x = st["q"][off[b] + i:min(off[b] + i + 512, off[b + 1]), h * G:(h + 1) * G].double()
                s = torch.einsum("ngd,sd->ngs", x, k) * D ** -0.5
                s.masked_fill_(~see[i:i + x.shape[0]][:, None, :], -math.inf)
                out[off[b] + i:off[b] + i + x.shape[0], h * G:(h + 1) * G] = torch.softmax(s, -1) @ v
    return out
