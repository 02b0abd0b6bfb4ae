"""What is measured of the steps between a decoder's projections and its next
token: rotary positions and the write into a paged cache, attention over that
cache, beam selection over the logits, and the cache's pages.

Each as a plain form in elementary torch operations and as the framework's own
call (`own`):

  rotary     q, k turned by their positions (several axes), k and v written
             into a paged cache                                sgemv_rotary
  attention  one new token over the cache's pages              sgemv_attn_paged
  beam       the best continuations over beams and vocabulary  sgemv_beam_select
  fork       rows that take over their parents' pages, grow and
             copy what they share                              sgemv_pages_fork
  compact    used pages moved to the front of the pool         sgemv_pages_compact
"""
import math

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"f16": 2, "bf16": 2, "f32": 4, "e4m3": 1}
E4M3_MAX = 448.0


def _attention(name, B, Hq, Hkv, D, most, page, x, cache=None, least=1, window=0, softcap=0.0, lse=False,
               layout="tokens"):
    return {"name": name, "op": "attention", "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "most": most, "least": least,
            "page": page, "x": x, "cache": cache or x, "window": window, "softcap": softcap, "lse": lse,
            "layout": layout}


def _rotary(name, T, Hq, Hkv, D, rot, x, axes=1, adjacent=False, striped=False, cache=None, page=16, far=4096,
            layout="tokens"):
    return {"name": name, "op": "rotary", "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot, "x": x, "axes": axes,
            "adjacent": adjacent, "striped": striped, "cache": cache, "page": page, "far": far, "layout": layout}


def _beam(name, B, W, V, n, x, finished=False):
    return {"name": name, "op": "beam", "B": B, "W": W, "V": V, "n": n, "x": x, "finished": finished}


def _fork(name, rows, most, page, Hkv, D, layers, x, beams, grow=1):
    return {"name": name, "op": "fork", "rows": rows, "most": most, "page": page, "Hkv": Hkv, "D": D,
            "layers": layers, "x": x, "beams": beams, "grow": grow}


def _compact(name, rows, pages, page, Hkv, D, layers, x, used):
    return {"name": name, "op": "compact", "rows": rows, "pages": pages, "page": page, "Hkv": Hkv, "D": D,
            "layers": layers, "x": x, "used": used}


def listed():
    return [
        # one short conversation, the heads of an 8B layer: latency
        _attention("attention 1x640", 1, 32, 8, 128, 640, 16, "f16", least=640),
        # sixteen sequences of every length, one of them empty, the heads of a 70B layer
        _attention("attention 16 ragged to 32768", 16, 64, 8, 128, 32768, 64, "bf16", least=0),
        # a full batch of long contexts: the largest
        _attention("attention 48x24000", 48, 64, 8, 128, 24000, 64, "bf16", least=20011),
        # keys and values in 8 bits, pages that are no power of two, a window, a soft cap, odd head sizes and counts
        _attention("attention 7 windowed e4m3", 7, 20, 4, 96, 5000, 24, "f16", "e4m3", least=3, window=1500,
                   softcap=30.0, lse=True, layout="heads"),
        # one new token of an 8B layer: between the projection and the attention
        _rotary("rotary 1 token", 1, 32, 8, 128, 128, "f16", cache="f16"),
        # a long prompt with images: three axes, the heads of a 70B layer
        _rotary("rotary 16384 three axes", 16384, 64, 8, 128, 128, "bf16", axes=3, cache="bf16", page=64, far=20000),
        # part of each head turned, neighbours as pairs, axes dealt in turn, far positions, keys and values in 8 bits
        _rotary("rotary 777 partial e4m3", 777, 20, 4, 96, 48, "f16", axes=2, adjacent=True, striped=True,
                cache="e4m3", page=24, far=1000003),
        # four beams of one request
        _beam("beam 1x4x32003", 1, 4, 32003, 8, "f16"),
        # a batch of searches over a large vocabulary, some beams finished
        _beam("beam 48x8x100003", 48, 8, 100003, 16, "bf16", finished=True),
        # four beams change places and take one token each, one layer
        _fork("fork 4 rows", 4, 300, 16, 8, 128, 1, "f16", 4),
        # thirty-two searches of eight beams, four layers
        _fork("fork 256 rows", 256, 2000, 32, 8, 128, 4, "bf16", 8),
        # a pool after many requests have ended: a quarter of its pages move
        _compact("compact 1500 pages", 64, 1500, 64, 8, 128, 2, "bf16", 0.55),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "rotary", "beam", "fork", "compact"])
    x = rng.choice(["f16", "bf16"])
    D = rng.choice([64, 128, 128, 8 * rng.randint(3, 32)])
    Hkv = rng.choice([1, 2, 4, 8, 8, rng.randint(1, 12)])
    page = rng.choice([16, 16, 32, 64, 128, rng.randint(3, 100)])
    layout = rng.choice(["tokens", "tokens", "heads"])
    if op == "attention":
        group = rng.choice([1, 4, 4, 8, 8, rng.randint(1, 20)])
        B = _log_int(rng, 1, 128)
        most = _log_int(rng, 1, max(2, min(131072, 1000000000 // (B * Hkv * D))))
        ragged = rng.random() < 0.6
        return {"op": op, "B": B, "Hq": Hkv * group, "Hkv": Hkv, "D": D, "most": most,
                "least": rng.choice([0, 1, 1 + most // 10]) if ragged else most, "page": page, "x": x,
                "cache": rng.choice([x, x, "e4m3"]), "window": rng.choice([0, 0, 0, _log_int(rng, 1, most)]),
                "softcap": rng.choice([0.0, 0.0, 30.0]), "lse": rng.random() < 0.4, "layout": layout}
    if op == "rotary":
        Hq = Hkv * rng.choice([1, 4, 8, rng.randint(1, 8)])
        rot = D if rng.random() < 0.6 else 2 * rng.randint(3, D // 2)
        T = _log_int(rng, 1, max(1, 16384 * 72 * 128 // ((Hq + Hkv) * D)))
        # 8-bit caches are kept small: their values are written out whole
        small = T * Hkv * D < 1500000
        return {"op": op, "T": min(T, 40000), "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot, "x": rng.choice([x, x, "f32"]),
                "axes": rng.choice([1, 1, 2, 3, 3]), "adjacent": rng.random() < 0.4, "striped": rng.random() < 0.5,
                "cache": rng.choice([None, x, x] + (["e4m3"] if small else [])), "page": page,
                "far": _log_int(rng, 100, 10000000), "layout": layout}
    if op == "beam":
        W = rng.choice([1, 2, 4, 5, 8, 16])
        V = _log_int(rng, 300, 100003)
        B = _log_int(rng, 1, max(1, min(64, 48 * 8 * 100003 // (W * V))))
        return {"op": op, "B": B, "W": W, "V": V, "n": rng.choice([W, 2 * W]), "x": rng.choice([x, "f32"]),
                "finished": rng.random() < 0.5}
    layers = rng.choice([1, 2, 4])
    token = Hkv * D * layers * 2
    pages = _log_int(rng, 24, max(25, min(4000, 300000000 // (token * page))))
    if op == "fork":
        rows = min(_log_int(rng, 2, 256), max(2, pages // 6))
        beams = rng.choice([1, 2, 4, 8])
        most = max(2, min(8000, pages // (2 + rows) * page))
        return {"op": op, "rows": rows, "most": most, "page": page, "Hkv": Hkv, "D": D, "layers": layers, "x": x,
                "beams": beams, "grow": rng.choice([1, 1, 2, rng.randint(1, 9)])}
    return {"op": op, "rows": rng.randint(1, min(64, pages // 3)), "pages": pages, "page": page, "Hkv": Hkv, "D": D,
            "layers": layers, "x": x, "used": rng.choice([0.3, 0.55, 0.8])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _lengths(case):
    """Lengths of a batch: spread over their logarithm between `least` and
    `most`; a `least` of zero makes one sequence empty."""
    B, most, least = case["B"], case["most"], max(1, case["least"])
    if B == 1 or least == most:
        got = [most] * B
    else:
        got = [max(1, int(round(least * (most / least) ** (i / (B - 1))))) for i in range(B)]
    if case["least"] == 0 and B > 1:
        got[0] = 0
    return got


def _pool(gen, shape, t, layout):
    """A pool of pages as a [pages][page][heads][D] view of either layout, of
    normal values."""
    pages, page, heads, D = shape
    inner = (heads, page, D) if layout == "heads" else (page, heads, D)
    pool = torch.empty(pages, *inner, dtype=TYPES[t], device=gen.device)
    step = max(1, (1 << 27) // (page * heads * D))
    for p in range(0, pages, step):
        part = torch.randn(min(step, pages - p), *inner, generator=gen, device=gen.device)
        pool[p:p + step] = part.mul_(16.0).clamp_(-E4M3_MAX, E4M3_MAX) if t == "e4m3" else part
    return pool.transpose(1, 2) if layout == "heads" else pool


def _scales(gen, case):
    """What one unit of an 8-bit cache stands for, a factor for each head."""
    if case["cache"] != "e4m3":
        return None, None
    return tuple((0.05 + 0.03 * torch.rand(case["Hkv"], generator=gen, device=gen.device)) for _ in range(2))


def _attention_inputs(case, gen):
    s, dev, lens = dict(case), gen.device, _lengths(case)
    order = torch.randperm(len(lens), generator=gen, device=dev)
    s["lengths"] = torch.tensor(lens, dtype=torch.int32, device=dev)[order]
    B, page = case["B"], case["page"]
    per = [-(-n // page) for n in lens]
    width = max(per + [1])
    held = (s["lengths"].long() + page - 1) // page
    pages = sum(per) + 3
    ids = torch.randperm(pages, generator=gen, device=dev)
    col = torch.arange(width, device=dev)
    first = held.cumsum(0) - held
    table = torch.where(col < held[:, None], ids[(first[:, None] + col).clamp(max=pages - 1)], -1)
    s["table"] = table.to(torch.int32)
    s["k"] = _pool(gen, (pages, page, case["Hkv"], case["D"]), case["cache"], case["layout"])
    s["v"] = _pool(gen, (pages, page, case["Hkv"], case["D"]), case["cache"], case["layout"])
    s["k_scale"], s["v_scale"] = _scales(gen, case)
    q = torch.randn(B, case["Hq"], case["D"], generator=gen, device=dev) * (1.0 + 0.5 * torch.rand(
        case["D"], generator=gen, device=dev))
    s["q"] = q.to(TYPES[case["x"]])
    return s


def _sections(case):
    """Frequency pairs of each axis: a little more for the first."""
    pairs, axes = case["rot"] // 2, case["axes"]
    rest = [pairs // axes] * axes
    rest[0] += pairs - sum(rest)
    return rest


def _axis_of(case):
    """Axis of every pair: blocks, or dealt in turn while an axis has pairs
    left."""
    left = _sections(case)
    if not case["striped"]:
        return [a for a, n in enumerate(left) for _ in range(n)]
    got = []
    while sum(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                got.append(a)
    return got


def _rotary_inputs(case, gen):
    s, dev = dict(case), gen.device
    T, Hq, Hkv, D, t = case["T"], case["Hq"], case["Hkv"], case["D"], TYPES[case["x"]]
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=gen, device=dev).to(t)   # one projection's output
    s["q"], s["kt"], s["vt"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    first = torch.randint(0, max(1, case["far"] - T), (1,), generator=gen, device=dev)
    pos = (first + torch.arange(T, device=dev))[None].repeat(case["axes"], 1)
    if case["axes"] > 1:   # places of an image: rows and columns beside the time
        pos[1:] = first + torch.randint(0, 64, (case["axes"] - 1, T), generator=gen, device=dev)
    s["positions"] = pos.to(torch.int32)
    s["inv_freq"] = (500000.0 ** (-torch.arange(0, case["rot"], 2, device=dev, dtype=torch.float64) / case["rot"])).float()
    s["slots"] = None
    if case["cache"]:
        pages = -(-T // case["page"]) + 2
        slots = torch.randperm(pages * case["page"], generator=gen, device=dev)[:T].to(torch.int32)
        if T > 8:   # padding
            slots[torch.randint(0, T, (T // 8,), generator=gen, device=dev)] = -1
        s["slots"] = slots
        s["k"] = _pool(gen, (pages, case["page"], Hkv, D), case["cache"], case["layout"])
        s["v"] = _pool(gen, (pages, case["page"], Hkv, D), case["cache"], case["layout"])
        s["k_scale"], s["v_scale"] = _scales(gen, case)
    return s


def _beam_inputs(case, gen):
    s, dev = dict(case), gen.device
    B, W, V = case["B"], case["W"], case["V"]
    logits = torch.empty(B, W, V, dtype=TYPES[case["x"]], device=dev)
    for b in range(B):
        logits[b] = 2.5 * torch.randn(W, V, generator=gen, device=dev)
    logits[:, :, torch.randperm(V, generator=gen, device=dev)[:max(1, V // 50)]] = -math.inf   # forbidden tokens
    s["logits"] = logits
    s["scores"] = -20.0 * torch.rand(B, W, generator=gen, device=dev)
    s["done"] = None
    if case["finished"]:
        s["done"] = (torch.rand(B, W, generator=gen, device=dev) < 0.25).to(torch.uint8)
    s["end"] = V // 3
    return s


def _pools(case, gen, pages):
    def one():
        return torch.randn(case["layers"], pages, case["page"], case["Hkv"], case["D"], generator=gen,
                           device=gen.device, dtype=torch.float16).to(TYPES[case["x"]])
    return one(), one()


def _fork_inputs(case, gen):
    """Rows in groups of `beams` that share all but their last page or two."""
    s, dev, rows, page, beams = dict(case), gen.device, case["rows"], case["page"], case["beams"]
    width = -(-(case["most"] + case["grow"]) // page)
    table, lengths, taken = [], [], 0
    for g in range(0, rows, beams):
        n = max(1, int(round(case["most"] ** (0.4 + 0.6 * ((g // beams * 7) % 11) / 10))))
        held = -(-n // page)
        shared = list(range(taken, taken + max(0, held - 2)))
        taken += len(shared)
        for _ in range(min(beams, rows - g)):
            mine = held - len(shared)
            table.append(shared + list(range(taken, taken + mine)) + [-1] * (width - held))
            taken += mine
            lengths.append(n)
    pages = taken + 2 * rows * (1 + -(-case["grow"] // page)) + 3
    ids = torch.randperm(pages, generator=gen, device=dev)
    t = torch.tensor(table, device=dev)
    t = torch.where(t >= 0, ids[t.clamp(min=0)], -1)
    s["table"], s["lengths"] = t.to(torch.int32), torch.tensor(lengths, dtype=torch.int32, device=dev)
    s["refs"] = torch.bincount(torch.where(t >= 0, t, pages).reshape(-1), minlength=pages + 1)[:pages].to(torch.int32)
    pick = torch.randint(0, beams, (rows,), generator=gen, device=dev)
    group = torch.arange(rows, device=dev) // beams * beams
    parents = torch.minimum(group + pick, torch.tensor(rows - 1, device=dev)).to(torch.int32)
    if rows > 8:
        parents[torch.randint(0, rows, (1,), generator=gen, device=dev)] = -1   # a row that ends
    s["parents"] = parents
    s["grow_by"] = torch.where(parents >= 0, case["grow"], 0).to(torch.int32)
    s["kp"], s["vp"] = _pools(case, gen, pages)
    return s


def _compact_inputs(case, gen):
    s, dev, pages, rows = dict(case), gen.device, case["pages"], case["rows"]
    used = max(rows, int(case["used"] * pages))
    ids = torch.randperm(pages, generator=gen, device=dev)[:used]
    width = -(-used // rows) + 1
    flat = torch.full((rows * width,), -1, dtype=torch.int64, device=dev)
    i = torch.arange(used, device=dev)
    flat[i % rows * width + i // rows] = ids
    held = torch.bincount(i % rows, minlength=rows)
    s["table"] = flat.view(rows, width).to(torch.int32)
    s["lengths"] = (held * case["page"] - torch.randint(0, case["page"], (rows,), generator=gen, device=dev)).to(torch.int32)
    s["refs"] = torch.zeros(pages, dtype=torch.int32, device=dev).index_fill_(0, ids, 1)
    s["kp"], s["vp"] = _pools(case, gen, pages)
    return s


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"attention": _attention_inputs, "rotary": _rotary_inputs, "beam": _beam_inputs, "fork": _fork_inputs,
            "compact": _compact_inputs}[case["op"]](case, gen)


def prepare(case, seed):
    s = _inputs(case, seed)
    op, dev = case["op"], "cuda"
    if op == "attention":
        s["out"] = torch.empty_like(s["q"])
        s["lse_out"] = torch.empty(case["B"], case["Hq"], device=dev) if case["lse"] else None
    elif op == "rotary":
        s["q_out"] = torch.empty(case["T"], case["Hq"], case["D"], dtype=s["q"].dtype, device=dev)
        s["k_out"] = torch.empty(case["T"], case["Hkv"], case["D"], dtype=s["q"].dtype, device=dev)
    elif op == "beam":
        s["tokens"], s["parents"] = (torch.empty(case["B"], case["n"], dtype=torch.int32, device=dev) for _ in range(2))
        s["scores_out"] = torch.empty(case["B"], case["n"], device=dev)
    else:
        s["table_out"], s["refs_out"] = torch.empty_like(s["table"]), torch.empty_like(s["refs"])
        s["count"] = torch.empty(1, dtype=torch.int32, device=dev)
        n = case["rows"] if op == "fork" else case["pages"]
        s["pairs"] = torch.empty(n, 3, dtype=torch.int32, device=dev)
        if op == "fork":
            s["lengths_out"] = torch.empty_like(s["lengths"])
            s["slots_out"] = torch.empty(case["rows"], case["grow"], dtype=torch.int32, device=dev)
            s["status"] = torch.empty(2, dtype=torch.int32, device=dev)
    if own:
        from activation_sparse_bit_amd import sgemv
        s["lib"] = sgemv
        size = 0
        if op in ("attention", "rotary") and case["cache"]:
            s["kv"] = sgemv.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        if op == "attention":
            size = sgemv.sgemv_attn_workspace_bytes(case["B"], case["Hq"], case["Hkv"], case["D"])
        elif op == "beam":
            size = sgemv.sgemv_beam_workspace_bytes(case["B"], case["W"], case["V"], case["n"])
        elif op in ("fork", "compact"):
            s["caches"] = [sgemv.KVCache(k, v) for k, v in zip(s["kp"], s["vp"])]
            size = sgemv.sgemv_pages_workspace_bytes(case["rows"], s["table"].shape[1], s["refs"].shape[0])
        s["workspace"] = torch.zeros(max(size, 256), dtype=torch.uint8, device=dev)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _own(s):
    lib, op = s["lib"], s["op"]
    if op == "attention":
        lib.sgemv_attn_paged(s["q"], s["kv"], s["table"], s["lengths"], s["out"], s["workspace"], window=s["window"],
                             softcap=s["softcap"], lse=s["lse_out"])
        return {"out": s["out"], "lse": s["lse_out"]}
    if op == "rotary":
        if s["cache"]:
            lib.sgemv_rotary(s["q"], s["q_out"], s["positions"], s["inv_freq"], k=s["kt"], v=s["vt"], cache=s["kv"],
                             slots=s["slots"], sections=_sections(s), adjacent=s["adjacent"], striped=s["striped"])
            return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
        lib.sgemv_rotary(s["q"], s["q_out"], s["positions"], s["inv_freq"], k=s["kt"], k_out=s["k_out"],
                         sections=_sections(s), adjacent=s["adjacent"], striped=s["striped"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "beam":
        lib.sgemv_beam_select(s["logits"], s["scores"], s["tokens"], s["parents"], s["scores_out"], s["workspace"],
                              finished=s["done"], end_token=s["end"])
        return {"tokens": s["tokens"], "parents": s["parents"], "scores": s["scores_out"]}
    if op == "fork":
        lib.sgemv_pages_fork(s["table"], s["lengths"], s["refs"], s["table_out"], s["lengths_out"], s["refs_out"],
                             s["workspace"], page_size=s["page"], parents=s["parents"], grow=s["grow_by"],
                             slots=s["slots_out"], pairs=s["pairs"], count=s["count"], status=s["status"],
                             caches=s["caches"])
        return {"table": s["table_out"], "lengths": s["lengths_out"], "refs": s["refs_out"], "slots": s["slots_out"],
                "pairs": s["pairs"], "count": s["count"], "status": s["status"], "k": s["kp"], "v": s["vp"]}
    lib.sgemv_pages_compact(s["table"], s["lengths"], s["refs"], s["table_out"], s["refs_out"], s["workspace"],
                            page_size=s["page"], pairs=s["pairs"], count=s["count"], caches=s["caches"])
    return {"table": s["table_out"], "refs": s["refs_out"], "pairs": s["pairs"], "count": s["count"], "k": s["kp"],
            "v": s["vp"]}


def _plain_attention(s):
    B, Hq, Hkv, D, page = s["B"], s["Hq"], s["Hkv"], s["D"], s["page"]
    width = s["table"].shape[1]
    ids = s["table"].clamp(min=0).long().reshape(-1)
    k = s["k"][ids].reshape(B, width * page, Hkv, D).permute(0, 2, 3, 1).float()
    if s["k_scale"] is not None:
        k *= s["k_scale"][:, None, None]
    q = s["q"].float().reshape(B, Hkv, Hq // Hkv, D)
    p = torch.matmul(q, k) / math.sqrt(D)
    del k
    if s["softcap"]:
        p = s["softcap"] * torch.tanh(p / s["softcap"])
    token, n = torch.arange(width * page, device=q.device), s["lengths"][:, None]
    seen = token < n
    if s["window"]:
        seen = seen & (token >= n - s["window"])
    p = torch.where(seen[:, None, None], p, -math.inf)
    m = p.amax(-1, keepdim=True)
    p = torch.exp(p - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    v = s["v"][ids].reshape(B, width * page, Hkv, D).permute(0, 2, 1, 3).float()
    v = torch.where(seen[:, None, :, None], v, 0.0)
    if s["v_scale"] is not None:
        v *= s["v_scale"][:, None, None]
    out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    lse = (m + torch.log(total)).reshape(B, Hq) if s["lse"] else None
    return {"out": out.reshape(B, Hq, D).to(s["q"].dtype), "lse": lse}


def _plain_turn(x, cos, sin, rot, adjacent):
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if adjacent else (x[..., :rot // 2], x[..., rot // 2:rot])
    a, b = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((a, b), -1).flatten(-2) if adjacent else torch.cat((a, b), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_store(pool, x, scale, slots):
    if scale is not None:
        x = torch.clamp(x / scale[:, None], -E4M3_MAX, E4M3_MAX)
    keep, page = slots >= 0, pool.shape[1]
    at = slots[keep].long()
    pool[at // page, at % page] = x[keep].to(pool.dtype)
    return pool


def _plain_rotary(s):
    axis = torch.tensor(_axis_of(s), device=s["q"].device)
    angle = s["positions"].double()[axis].t() * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    q = _plain_turn(s["q"], cos, sin, s["rot"], s["adjacent"]).to(s["q"].dtype)
    k = _plain_turn(s["kt"], cos, sin, s["rot"], s["adjacent"])
    if not s["cache"]:
        return {"q": q, "k": k.to(s["kt"].dtype)}
    return {"q": q, "k": _plain_store(s["k"], k, s["k_scale"], s["slots"]),
            "v": _plain_store(s["v"], s["vt"].float(), s["v_scale"], s["slots"])}


def _plain_beam(s):
    B, W, V, n = s["B"], s["W"], s["V"], s["n"]
    x = s["logits"].double()
    m = x.amax(-1, keepdim=True)
    x -= m + torch.log(torch.exp(x - m).sum(-1, keepdim=True))
    x += s["scores"].double()[..., None]
    if s["done"] is not None:
        done = s["done"].bool()[..., None]
        end = torch.arange(V, device=x.device) == s["end"]
        x = torch.where(done, torch.where(end, s["scores"].double()[..., None], -math.inf), x)
    best, at = torch.sort(x.reshape(B, W * V), dim=-1, descending=True, stable=True)
    best, at = best[:, :n], at[:, :n]
    none = best == -math.inf
    return {"tokens": torch.where(none, -1, at % V).int(), "parents": torch.where(none, -1, at // V).int(),
            "scores": best.float()}


def _plain_fork(s):
    rows, page, P = s["rows"], s["page"], s["refs"].shape[0]
    table, lengths, grow, dev = s["table"].long(), s["lengths"].long(), s["grow_by"].long(), s["table"].device
    width, row = table.shape[1], torch.arange(rows, device=dev)
    col = torch.arange(width, device=dev)
    parent = s["parents"].long()
    alive = (parent >= 0) & (parent < rows)
    parent = torch.where(alive, parent, 0)
    n = torch.where(alive, lengths[parent], 0)
    held = (n + page - 1) // page
    new = torch.where(col < held[:, None], table[parent], -1)
    old = torch.where(col < ((lengths + page - 1) // page)[:, None], table, -1)
    one = torch.ones(rows * width, dtype=torch.long, device=dev)
    refs = torch.cat((s["refs"].long(), torch.zeros(1, dtype=torch.long, device=dev)))
    refs.index_add_(0, torch.where(new >= 0, new, P).reshape(-1), one)
    refs.index_add_(0, torch.where(old >= 0, old, P).reshape(-1), -one)
    refs[P] = 1
    # a shared last page is copied by every growing row, but by the last one where no one else holds it
    partial = (grow > 0) & (n % page > 0)
    at = (n // page).clamp(max=width - 1)
    last = torch.where(partial, new.gather(1, at[:, None])[:, 0], P)
    holders = torch.zeros(P + 1, dtype=torch.long, device=dev).index_add_(0, last, one[:rows])
    highest = torch.full((P + 1,), -1, dtype=torch.long, device=dev).scatter_reduce_(0, last, row, "amax")
    copied = partial & (refs[last] > 1) & ~((holders[last] == refs[last]) & (highest[last] == row))
    held_then = (n + grow + page - 1) // page
    need = copied.long() + held_then - held
    first = need.cumsum(0) - need
    free = torch.sort((refs > 0).int(), stable=True).indices
    missing = (need.sum() - (refs == 0).sum()).clamp(min=0)
    fresh = (col >= held[:, None]) & (col < held_then[:, None])
    fresh_id = free[(first[:, None] + copied.long()[:, None] + col - held[:, None]).clamp(0, P - 1)]
    new = torch.where(fresh, fresh_id, new)
    source, target = torch.where(copied, last, -1), torch.where(copied, free[first.clamp(max=P - 1)], -1)
    new = torch.where(copied[:, None] & (col == at[:, None]), target[:, None], new)
    refs.index_add_(0, torch.where(copied, last, P), -copied.long())
    refs.index_add_(0, torch.where(copied, target, P), copied.long())
    refs.index_add_(0, torch.where(fresh, fresh_id, P).reshape(-1), fresh.long().reshape(-1))
    j = torch.arange(s["slots_out"].shape[1], device=dev)
    token = n[:, None] + j
    slot = new.gather(1, (token // page).clamp(max=width - 1)) * page + token % page
    slots = torch.where(j < grow[:, None], slot, -1)
    pairs = torch.full((rows, 3), -1, dtype=torch.long, device=dev)
    who = copied.nonzero()[:, 0]
    source, target, tokens = source[who], target[who], (n % page)[who]
    pairs[:len(who)] = torch.stack((source, target, tokens), 1)
    within = (torch.arange(page, device=dev) < tokens[:, None])[None, :, :, None, None]
    for pool in (s["kp"], s["vp"]):
        pool[:, target] = torch.where(within, pool[:, source], pool[:, target])
    return {"table": new.int(), "lengths": (n + grow).int(), "refs": refs[:P].int(), "slots": slots.int(),
            "pairs": pairs.int(), "count": copied.sum().int().reshape(1),
            "status": torch.stack((missing, torch.zeros_like(missing))).int(), "k": s["kp"], "v": s["vp"]}


def _plain_compact(s):
    P, page = s["refs"].shape[0], s["page"]
    used, ids = s["refs"] > 0, torch.arange(P, device=s["refs"].device)
    front = ids < used.sum()
    source, target = (used & ~front).nonzero()[:, 0], (~used & front).nonzero()[:, 0]
    to = ids.clone()
    to[source] = target
    refs = s["refs"].clone()
    refs[target] = s["refs"][source]
    refs[source] = 0
    col = torch.arange(s["table"].shape[1], device=ids.device)
    held = (s["lengths"].long() + page - 1) // page
    table = torch.where(col < held[:, None], to[s["table"].clamp(min=0).long()], -1)
    pairs = torch.full((P, 3), -1, dtype=torch.long, device=ids.device)
    pairs[:len(source)] = torch.stack((source, target, torch.full_like(source, page)), 1)
    for pool in (s["kp"], s["vp"]):
        pool[:, target] = pool[:, source]
    return {"table": table.int(), "refs": refs, "pairs": pairs.int(),
            "count": (used & ~front).sum().int().reshape(1), "k": s["kp"], "v": s["vp"]}


def run(s):
    if own:
        return _own(s)
    return {"attention": _plain_attention, "rotary": _plain_rotary, "beam": _plain_beam, "fork": _plain_fork,
            "compact": _plain_compact}[s["op"]](s)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _fork_moves(case):
    """Tokens copied and pages held, about: a page's part for most rows, since beams share their parents."""
    lens = [max(1, int(round(case["most"] ** (0.4 + 0.6 * ((g // case["beams"] * 7) % 11) / 10))))
            for g in range(0, case["rows"], case["beams"])]
    share = 0.0 if case["beams"] == 1 else 0.6
    tokens = sum(n % case["page"] for n in lens) * min(case["beams"], case["rows"]) * share
    held = sum(-(-n // case["page"]) for n in lens) * min(case["beams"], case["rows"])
    return tokens, held


def work(case):
    op = case["op"]
    if op == "attention":
        seen = sum(min(n, case["window"]) if case["window"] else n for n in _lengths(case))
        held = seen // case["page"] + case["B"]
        heads = case["B"] * case["Hq"]
        return {"bytes": 2 * seen * case["Hkv"] * case["D"] * BYTES[case["cache"]] + 4 * held + 4 * case["B"]
                + 2 * heads * case["D"] * BYTES[case["x"]] + (4 * heads if case["lse"] else 0),
                "flops": 4 * seen * case["Hq"] * case["D"]}
    if op == "rotary":
        T, each = case["T"], BYTES[case["x"]]
        kept = BYTES[case["cache"]] * 2 if case["cache"] else each
        values = case["T"] * case["D"]
        read = values * each * (case["Hq"] + case["Hkv"] * (2 if case["cache"] else 1))
        written = values * (each * case["Hq"] + kept * case["Hkv"])
        return {"bytes": read + written + 4 * T * (case["axes"] + bool(case["cache"])),
                "flops": 3 * T * (case["Hq"] + case["Hkv"]) * case["rot"]}
    if op == "beam":
        all_ = case["B"] * case["W"] * case["V"]
        return {"bytes": all_ * BYTES[case["x"]] + 4 * case["B"] * (case["W"] + 3 * case["n"]), "flops": 4 * all_}
    token = 2 * case["layers"] * case["Hkv"] * case["D"] * BYTES[case["x"]]
    if op == "fork":
        tokens, held = _fork_moves(case)
        return {"bytes": 2 * tokens * token + 16 * held + 20 * case["rows"], "flops": 0}
    used = int(case["used"] * case["pages"])
    moved = used * (case["pages"] - used) // case["pages"]
    return {"bytes": 2 * moved * case["page"] * token + 8 * used + 8 * case["pages"], "flops": 0}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_attention(s):
    B, Hq, Hkv, D, page = s["B"], s["Hq"], s["Hkv"], s["D"], s["page"]
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device=s["q"].device)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=s["q"].device)
    for b, n in enumerate(s["lengths"].tolist()):
        if n == 0:
            continue
        ids = s["table"][b, :-(-n // page)].long()
        lo = max(0, n - s["window"]) if s["window"] else 0
        for h in range(Hkv):
            k = s["k"][ids, :, h].double().reshape(-1, D)[lo:n]
            v = s["v"][ids, :, h].double().reshape(-1, D)[lo:n]
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            z = torch.mm(k, s["q"][b, heads].double().t().contiguous()) * D ** -0.5
            if s["softcap"]:
                z = torch.tanh(z / s["softcap"]) * s["softcap"]
            lse[b, heads] = torch.logsumexp(z, 0)
            out[b, heads] = torch.mm(torch.softmax(z, 0).t().contiguous(), v)
    return {"out": out, "lse": lse if s["lse"] else None}


def _exact_rotary(s):
    rot, D, dev = s["rot"], s["D"], s["q"].device
    turn = torch.view_as_complex(torch.zeros(s["T"], D, 2, dtype=torch.float64, device=dev))
    turn += 1.0
    pair = torch.full((D,), -1, dtype=torch.long, device=dev)   # the value that each one turns with
    for i, axis in enumerate(_axis_of(s)):
        a, b = (2 * i, 2 * i + 1) if s["adjacent"] else (i, i + rot // 2)
        angle = s["positions"][axis].double() * s["inv_freq"][i].double()
        turn[:, a], turn[:, b] = torch.polar(torch.ones_like(angle), angle), torch.polar(torch.ones_like(angle), -angle)
        pair[a], pair[b] = b, a
    pair = torch.where(pair < 0, torch.arange(D, device=dev), pair)

    def turned(x):   # with w = cos + i sin for the first of a pair, its conjugate for the second
        x = x.double()
        return x * turn.real[:, None] - x[..., pair] * turn.imag[:, None]

    def stored(pool, x, scale):
        pool, x = pool.double(), x if scale is None else (x / scale.double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        keep = (s["slots"] >= 0).nonzero()[:, 0]
        at = s["slots"][keep].long()
        pool[torch.div(at, s["page"], rounding_mode="floor"), at % s["page"]] = x[keep]
        return pool

    got = {"q": turned(s["q"]), "k": turned(s["kt"])}
    if s["cache"]:
        got["k"] = stored(s["k"], got["k"], s["k_scale"])
        got["v"] = stored(s["v"], s["vt"].double(), s["v_scale"])
    return got


def _exact_beam(s):
    B, W, V, n = s["B"], s["W"], s["V"], s["n"]
    got = {"tokens": [], "parents": [], "scores": []}
    far = torch.arange(W * V, device=s["logits"].device)
    for b in range(B):
        z = torch.log_softmax(s["logits"][b].double(), -1) + s["scores"][b].double()[:, None]
        if s["done"] is not None:
            for w in s["done"][b].nonzero()[:, 0].tolist():
                z[w] = -math.inf
                z[w, s["end"]] = s["scores"][b, w].double()
        z, scores, at = z.reshape(-1), [], []
        for _ in range(n):
            top = z.max()
            first = torch.where(z == top, far, W * V).min()
            at.append(torch.where(top == -math.inf, -1, first))
            scores.append(top)
            z = torch.where(far == first, -math.inf, z)
        at = torch.stack(at)
        got["tokens"].append(torch.where(at < 0, -1, at % V).int())
        got["parents"].append(torch.where(at < 0, -1, at // V).int())
        got["scores"].append(torch.stack(scores))
    return {k: torch.stack(v) for k, v in got.items()}


def exact(case, seed):
    if case["op"] in ("fork", "compact"):   # whole numbers and copies
        return None
    s = _inputs(case, seed)
    return {"attention": _exact_attention, "rotary": _exact_rotary, "beam": _exact_beam}[case["op"]](s)
