"""Cases of the cache operators: what serving with a quantised key/value cache runs next to the
quantised linear layers.

  rope    rotary positions of queries and keys, and the gradient through them
  store   keys and values of new tokens written into the paged cache as codes and read back
  attend  attention of drafted tokens (a tree, a chain, or one token) over that cache

Definitions (row x of head dimension d):
  codes   z = R x (RPBH: gather, signs, blocks of a normalised Hadamard matrix), s = |z|,
          code_i = number of unit boundaries <= z_i sqrt(d) / (s + 1e-8)
  values  x_hat = s / sqrt(d) * R^T centroid[code]
  attend  o = sum_t p_t v_hat_t, p = softmax over the visible t of scale * q . k_hat_t;
          node i of a sequence sees its whole prefix and the nodes j with bit j of its mask
  rope    pair (a, b) -> amplitude * (a cos - b sin, a sin + b cos), angle = position * freq_i

`own` selects the framework's calls; otherwise `run` computes the plain form with elementary
torch operations in 32 bits (angles in 64).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-8


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
def listed():
    rope = lambda name, **k: {"name": name, "op": "rope", **k}      # noqa: E731
    store = lambda name, **k: {"name": name, "op": "store", **k}    # noqa: E731
    attend = lambda name, **k: {"name": name, "op": "attend", **k}  # noqa: E731
    return [
        # the queries and keys of one decoding step of 8 sequences, far into a scaled context
        rope("rope_step", T=8, hq=32, hk=8, d=128, rot=128, layout="half", scaling="yarn",
             factor=4.0, dtype="bf16", inverse=False, far=131072),
        # a prompt chunk with positions on half of each head, in adjacent pairs
        rope("rope_chunk", T=8192, hq=32, hk=8, d=128, rot=64, layout="interleaved",
             scaling="plain", factor=1.0, dtype="bf16", inverse=False, far=8192),
        # a training step's gradients of a ragged batch, in fp32, back through the positions
        rope("rope_grad", T=4099, hq=24, hk=24, d=128, rot=128, layout="half",
             scaling="linear", factor=2.0, dtype="f32", inverse=True, far=32768),
        # one decoding step of 8 sequences with 8 key/value heads
        store("store_step", T=8, heads=8, d=128, h=128, bits=4, page=16, dtype="bf16", pad=0),
        # a ragged prompt chunk; the batch's last rows are padding
        store("store_chunk", T=2011, heads=8, d=128, h=64, bits=4, page=16, dtype="bf16",
              pad=11),
        # wide heads in two-bit codes, fp16
        store("store_wide", T=5003, heads=4, d=256, h=128, bits=2, page=64, dtype="f16", pad=3),
        # every key and value of a video transformer's layer (40 heads, one 480p clip), 8 bits
        store("store_video", T=32760, heads=40, d=128, h=128, bits=8, page=64, dtype="bf16",
              pad=0),
        # one sequence, one token: latency
        attend("decode_one", B=1, nodes=1, hq=32, hk=8, d=128, h=128, bits=4, page=16, lo=4096,
               hi=4096, tree=False, dtype="bf16"),
        # a batch of single tokens over contexts of all lengths
        attend("decode_batch", B=64, nodes=1, hq=32, hk=8, d=128, h=128, bits=4, page=16, lo=37,
               hi=8191, tree=False, dtype="bf16"),
        # one query head per key head, three-bit codes, fp16
        attend("decode_mha", B=8, nodes=1, hq=40, hk=40, d=128, h=64, bits=3, page=32, lo=900,
               hi=3001, tree=False, dtype="f16"),
        # drafted trees of a batch, eight-bit codes
        attend("tree_batch", B=16, nodes=61, hq=32, hk=8, d=128, h=128, bits=8, page=64, lo=129,
               hi=4095, tree=True, dtype="bf16"),
        # a drafted tree at the end of a long context
        attend("tree_long", B=2, nodes=31, hq=32, hk=8, d=128, h=128, bits=4, page=64,
               lo=131001, hi=131072, tree=True, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "store", "attend"])
    d = rng.choice([128, 128, 256])
    if op == "rope":
        hk = rng.choice([1, 2, 5, 8, 24])
        return {"op": op, "T": _log(rng, 1, 4096), "hq": hk * rng.choice([1, 2, 4]), "hk": hk,
                "d": d, "rot": rng.choice([d, d // 2, 32]),
                "layout": rng.choice(["half", "interleaved"]),
                "scaling": rng.choice(["plain", "linear", "ntk", "yarn"]),
                "factor": rng.choice([2.0, 4.0, 8.0]), "dtype": rng.choice(["bf16", "f16", "f32"]),
                "inverse": rng.random() < 0.5, "far": _log(rng, 128, 1000000)}
    h = rng.choice([32, 64, 128])
    bits = rng.choice([2, 3, 4, 6, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "store":
        T = _log(rng, 1, 8192)
        return {"op": op, "T": T, "heads": rng.choice([1, 2, 5, 8, 12, 40]), "d": d, "h": h,
                "bits": bits, "page": page, "dtype": rng.choice(["bf16", "f16", "f32"]),
                "pad": rng.choice([0, 0, min(7, T - 1)])}
    hk = rng.choice([1, 2, 4, 8, 12])
    B = _log(rng, 1, 64)
    nodes, group = rng.choice([1, 1, 2, 7, 16, 33, 64]), rng.choice([1, 2, 4, 7])
    most = min(2000000, 240000000 // (nodes * group)) // (B * hk * (d // 128))   # cost
    hi = _log(rng, 1, max(1, min(65536, most)))
    return {"op": op, "B": B, "nodes": nodes, "hq": hk * group, "hk": hk,
            "d": d, "h": h, "bits": bits, "page": page, "lo": rng.randint(0, hi), "hi": hi,
            "tree": nodes > 1 and rng.random() < 0.7, "dtype": rng.choice(["bf16", "f16"])}


def _prefixes(case):
    """Cached tokens before the drafted ones, spread evenly over [lo, hi]."""
    B = case["B"]
    if B == 1:
        return [case["hi"]]
    return [case["lo"] + (case["hi"] - case["lo"]) * i // (B - 1) for i in range(B)]


def work(case):
    d = case["d"]
    if case["op"] == "rope":
        size = 4 if case["dtype"] == "f32" else 2
        n = case["T"] * (case["hq"] + case["hk"]) * d
        return {"bytes": 2 * n * size + 8 * case["T"], "flops": 3 * n * case["rot"] / d}
    if case["op"] == "store":
        size = 4 if case["dtype"] == "f32" else 2
        out = 2
        rows = 2 * case["T"] * case["heads"]
        # written: rows read, codes and norms written; read back: codes, norms read, rows written
        return {"bytes": rows * (d * (size + out) + 2 * (d * case["bits"] // 8 + 4)),
                "flops": rows * d * 2 * math.log2(case["h"])}
    tokens = sum(_prefixes(case)) + case["B"] * case["nodes"]
    rows = case["B"] * case["nodes"] * case["hq"] * d
    pairs = case["nodes"] * case["hq"] * tokens
    return {"bytes": 2 * tokens * case["hk"] * (d * case["bits"] // 8 + 4) + 4 * rows,
            "flops": 4 * pairs * d}


# ---------------------------------------------------------------------------------------
# tables: the rotation and the codebook, from their definitions
# ---------------------------------------------------------------------------------------
def _rpbh(d, seed=0):
    """SplitMix64 -> Fisher-Yates permutation and signs."""
    mask, state = (1 << 64) - 1, seed

    def draw64():
        nonlocal state
        state = (state + 0x9E3779B97F4A7C15) & mask
        z = state
        z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & mask
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & mask
        return z ^ (z >> 31)

    perm = list(range(d))
    for i in range(d - 1, 0, -1):
        n = i + 1
        r = draw64()
        while r >= (1 << 64) - (1 << 64) % n:
            r = draw64()
        perm[i], perm[r % n] = perm[r % n], perm[i]
    sign = [-1.0 if draw64() >> 63 else 1.0 for _ in range(d)]
    return perm, sign


def _hadamard(h):
    m = np.ones((1, 1))
    while m.shape[0] < h:
        m = np.block([[m, m], [m, -m]])
    return m


_books = {}


def _codebook(bits):
    """Unit Lloyd-Max quantiser of N(0, 1): centroids and boundaries (Newton on the boundaries
    t_j = (c_j + c_{j+1}) / 2 with c_j the mean of its cell)."""
    if bits in _books:
        return _books[bits]
    L = 1 << bits
    pdf = lambda x: np.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)              # noqa: E731
    tail = np.vectorize(lambda x: 0.5 * math.erfc(x / math.sqrt(2)), otypes=[float])

    def cells(t):
        a, b = np.concatenate([[-np.inf], t]), np.concatenate([t, [np.inf]])
        lo, hi = np.where(a + b < 0, -b, a), np.where(a + b < 0, -a, b)        # the tail's side
        P = tail(lo) - tail(hi)
        fa, fb = pdf(a), pdf(b)
        mu = (fa - fb) / P
        da = np.where(np.isfinite(a), fa * (mu - np.where(np.isfinite(a), a, 0)) / P, 0)
        db = np.where(np.isfinite(b), fb * (np.where(np.isfinite(b), b, 0) - mu) / P, 0)
        return mu, da, db

    # cells of equal mass under the cube root of the density: N(0, 3)
    q = np.arange(1, L) / L
    t = np.array([_normal_quantile(v) for v in q]) * math.sqrt(3)
    for _ in range(60):
        mu, da, db = cells(t)
        f = t - 0.5 * (mu[:-1] + mu[1:])
        J = np.diag(1 - 0.5 * (db[:-1] + da[1:]))
        J -= np.diag(0.5 * da[1:-1], -1) + np.diag(0.5 * db[1:-1], 1) if L > 2 else 0
        step = np.linalg.solve(J, f)
        new = t - step
        while np.any(np.diff(new) <= 0):
            step = step / 2
            new = t - step
        t = new
        if np.abs(step).max() < 1e-14:
            break
    t = 0.5 * (t - t[::-1])
    c = cells(t)[0]
    c = 0.5 * (c - c[::-1])
    _books[bits] = (c, t)
    return c, t


def _normal_quantile(p):
    lo, hi = -9.0, 9.0
    for _ in range(80):
        m = 0.5 * (lo + hi)
        if 0.5 * math.erfc(-m / math.sqrt(2)) < p:
            lo = m
        else:
            hi = m
    return 0.5 * (lo + hi)


def _tables(case):
    d, h = case["d"], case["h"]
    perm, sign = _rpbh(d)
    c, t = _codebook(case["bits"])
    f = lambda a: torch.tensor(np.asarray(a), dtype=torch.float64, device="cuda")    # noqa: E731
    return {"perm": torch.tensor(perm, device="cuda"), "sign": f(sign), "had": f(_hadamard(h)),
            "cent": f(c), "bound": f(t)}


def _freq(case):
    """Frequencies (radians a position) and amplitude of the scaled forms, in 64 bits."""
    rot, factor, base = case["rot"], case["factor"], 10000.0
    i = np.arange(0, rot, 2, dtype=np.float64) / rot
    if case["scaling"] == "ntk":
        base = base * factor ** (rot / (rot - 2))
    freq = base ** -i
    if case["scaling"] == "linear":
        freq = freq / factor
    if case["scaling"] != "yarn":
        return freq, 1.0
    # turns that a pair makes over the original length: 32 and more stay, 1 and fewer are scaled
    at = lambda turns: rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    lo, hi = max(math.floor(at(32)), 0), min(math.ceil(at(1)), rot - 1)
    ramp = np.clip((np.arange(rot // 2) - lo) / max(hi - lo, 1e-3), 0, 1)
    return freq / factor * ramp + freq * (1 - ramp), 0.1 * math.log(factor) + 1.0


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"rope": _prepare_rope, "store": _prepare_store, "attend": _prepare_attend}[
        case["op"]](case, g, seed)


def _prepare_rope(case, g, seed):
    T, d, dt = case["T"], case["d"], DTYPES[case["dtype"]]
    freq, amp = _freq(case)
    s = {"case": case,
         "q": _normal(g, T, case["hq"], d).to(dt), "k": _normal(g, T, case["hk"], d).to(dt),
         "pos": torch.randint(0, case["far"], (T,), generator=g, device="cuda"),
         "freq": torch.tensor(freq, device="cuda"), "amp": amp}
    if own:
        from calibration_free_bit_b200 import oq
        s["rope"] = oq.oq_build_rope(case["rot"], layout=case["layout"], theta=10000.0,
                                     scaling=case["scaling"], factor=case["factor"],
                                     original_len=4096)
    return s


def _handles(oq, case, s):
    s["rpbh"] = oq.oq_build_rpbh(case["d"], case["h"], 0)
    s["book"] = oq.oq_lloyd_max(case["d"], case["bits"])


def _prepare_store(case, g, seed):
    T, H, d, P, dt = case["T"], case["heads"], case["d"], case["page"], DTYPES[case["dtype"]]
    pages = -(-T // P) + 2
    order = torch.randperm(pages, generator=g, device="cuda")
    t = torch.arange(T, device="cuda")
    slots = order[t // P] * P + t % P
    if case["pad"]:
        slots[T - case["pad"]:] = -1
    # keys carry a few loud channels, as a layer's keys do; the rows' sizes vary by token
    loud = torch.where(torch.rand(H, d, generator=g, device="cuda") < 0.02, 8.0, 1.0)
    size = torch.exp(0.4 * _normal(g, T, H, 1))
    s = {"case": case, "tables": _tables(case), "slots": slots,
         "k": (_normal(g, T, H, d) * loud * size).to(dt), "v": _normal(g, T, H, d).to(dt),
         "kc": torch.zeros(pages, H, P, d * case["bits"] // 8, dtype=torch.uint8, device="cuda"),
         "kn": torch.zeros(pages, H, P, device="cuda")}
    s["vc"], s["vn"] = torch.zeros_like(s["kc"]), torch.zeros_like(s["kn"])
    if own:
        from calibration_free_bit_b200 import oq
        _handles(oq, case, s)
        s["cache"] = oq.KVCache(s["kc"], s["vc"], s["kn"], s["vn"], bits=case["bits"])
    return s


def _random_codes(g, rows, case, bound):
    """Packed codes of normal rows, a block of rows at a time."""
    d, bits, out = case["d"], case["bits"], []
    for a in range(0, rows, 1 << 20):
        n = min(1 << 20, rows - a)
        out.append(_pack(torch.bucketize(_normal(g, n, d), bound, right=True), bits))
    return torch.cat(out)


def _prepare_attend(case, g, seed):
    B, n, hk, d, P = case["B"], case["nodes"], case["hk"], case["d"], case["page"]
    rng = np.random.default_rng(seed)
    prefix = np.array(_prefixes(case))
    rng.shuffle(prefix)
    need = -(-(prefix + n) // P)
    total = int(need.sum()) + 3
    order = rng.permutation(total)
    table = np.full((B, int(need.max()) + 1), -1, dtype=np.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    tables = _tables(case)
    bound = tables["bound"].float()
    rows = total * hk * P
    shape = (total, hk, P)
    s = {"case": case, "tables": tables,
         "kc": _random_codes(g, rows, case, bound).view(*shape, -1),
         "vc": _random_codes(g, rows, case, bound).view(*shape, -1),
         "kn": math.sqrt(d) * torch.exp(0.3 * _normal(g, *shape)),
         "vn": math.sqrt(d) * torch.exp(0.3 * _normal(g, *shape)),
         "q": (2 * _normal(g, B * n, case["hq"], d)).to(DTYPES[case["dtype"]]),
         "start": torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda"),
         "prefix": torch.tensor(prefix, dtype=torch.int32, device="cuda"),
         "table": torch.tensor(table, device="cuda"), "mask": None,
         "scale": 1 / math.sqrt(d)}
    if case["tree"]:
        # each drafted token continues one of the eight before it, or starts a branch
        words = np.zeros((B, n), dtype=np.uint64)
        parent = rng.integers(-1, 8, size=(B, n))
        for b in range(B):
            for i in range(n):
                up = i - 1 - int(parent[b, i])
                words[b, i] = np.uint64(1 << i) | (words[b, up] if 0 <= up < i else np.uint64(0))
        s["mask"] = torch.tensor(words.reshape(-1).view(np.int64), device="cuda")
    if own:
        from calibration_free_bit_b200 import oq
        _handles(oq, case, s)
        s["cache"] = oq.KVCache(s["kc"], s["vc"], s["kn"], s["vn"], bits=case["bits"])
    return s


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------
def run(state):
    return {"rope": _run_rope, "store": _run_store, "attend": _run_attend}[
        state["case"]["op"]](state)


def _run_rope(s):
    if own:
        from calibration_free_bit_b200 import oq
        q, k = oq.oq_apply_rope(s["rope"], s["q"], s["pos"], k=s["k"],
                                inverse=s["case"]["inverse"])
        return {"q": q, "k": k}
    c = s["case"]
    angle = s["pos"].double()[:, None] * s["freq"]
    cos = (s["amp"] * angle.cos()).float()[:, None]
    sin = (s["amp"] * angle.sin()).float()[:, None]
    if c["inverse"]:
        sin = -sin
    return {"q": _rope_plain(s["q"], cos, sin, c), "k": _rope_plain(s["k"], cos, sin, c)}


def _rope_plain(x, cos, sin, c):
    y = x.float()
    rot = c["rot"]
    head, rest = y[..., :rot], y[..., rot:]
    if c["layout"] == "half":
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([turned, rest], -1).to(x.dtype)


def _pack(codes, bits):
    """Codes [..., d] -> bytes [..., d * bits / 8], least significant bit first."""
    per = 8 // math.gcd(bits, 8)                   # codes in a whole number of bytes
    shift = bits * torch.arange(per, device=codes.device)
    word = (codes.view(*codes.shape[:-1], -1, per).to(torch.int32) << shift.int()).sum(-1)
    byte = torch.arange(per * bits // 8, device=codes.device).int() * 8
    return ((word[..., None] >> byte) & 255).to(torch.uint8).flatten(-2)


def _unpack(packed, bits):
    per = 8 // math.gcd(bits, 8)
    nb = per * bits // 8
    byte = torch.arange(nb, device=packed.device).int() * 8
    word = (packed.view(*packed.shape[:-1], -1, nb).to(torch.int32) << byte).sum(-1)
    shift = bits * torch.arange(per, device=packed.device)
    return ((word[..., None] >> shift.int()) & ((1 << bits) - 1)).flatten(-2)


def _rotate(x, tab):
    had = tab["had"].to(x.dtype)
    h = had.shape[0]
    y = x[..., tab["perm"]] * tab["sign"].to(x.dtype)
    return (y.unflatten(-1, (-1, h)) @ had).flatten(-2) / math.sqrt(h)


def _rotate_back(z, tab):
    had = tab["had"].to(z.dtype)
    h = had.shape[0]
    y = (z.unflatten(-1, (-1, h)) @ had).flatten(-2) / math.sqrt(h) * tab["sign"].to(z.dtype)
    return y[..., torch.argsort(tab["perm"])]


def _values(codes, norms, tab):
    """Rows that codes [..., bytes] and norms [...] stand for, in the norms' type."""
    bits = int(math.log2(tab["cent"].numel()))
    u = tab["cent"].to(norms.dtype)[_unpack(codes, bits)]
    return _rotate_back(u, tab) * (norms / math.sqrt(u.shape[-1]))[..., None]


def _write_plain(x, codes, norms, s):
    c, tab = s["case"], s["tables"]
    z = _rotate(x.float(), tab)
    norm = z.square().sum(-1).sqrt()
    u = z / (norm[..., None] + EPS) * math.sqrt(c["d"])
    packed = _pack(torch.bucketize(u, tab["bound"].float(), right=True), c["bits"])
    kept = s["slots"] >= 0
    page, at = s["slots"][kept] // c["page"], s["slots"][kept] % c["page"]
    codes[page, :, at] = packed[kept]
    norms[page, :, at] = norm[kept]


def _read_plain(codes, norms, s, dtype):
    c = s["case"]
    kept = s["slots"] >= 0
    slot = s["slots"].clamp(min=0)
    page, at = slot // c["page"], slot % c["page"]
    x = _values(codes[page, :, at], norms[page, :, at], s["tables"])
    return torch.where(kept[:, None, None], x, 0.0).to(dtype)


def _run_store(s):
    dt = torch.float16 if s["case"]["dtype"] == "f16" else torch.bfloat16
    if own:
        from calibration_free_bit_b200 import oq
        oq.oq_kv_write(s["rpbh"], s["book"], s["cache"], s["k"], s["v"], s["slots"])
        k, v = oq.oq_kv_read(s["rpbh"], s["book"], s["cache"], s["slots"], out_dtype=dt)
        return {"k": k, "v": v, "k_norms": s["kn"], "v_norms": s["vn"]}
    _write_plain(s["k"], s["kc"], s["kn"], s)
    _write_plain(s["v"], s["vc"], s["vn"], s)
    return {"k": _read_plain(s["kc"], s["kn"], s, dt), "v": _read_plain(s["vc"], s["vn"], s, dt),
            "k_norms": s["kn"], "v_norms": s["vn"]}


def _run_attend(s):
    c = s["case"]
    if own:
        from calibration_free_bit_b200 import oq
        return oq.oq_kv_attend(s["rpbh"], s["book"], s["cache"], s["q"], s["start"], s["prefix"],
                               s["table"], max_nodes=c["nodes"], tree_mask=s["mask"],
                               scale=s["scale"])
    B, n, hk, P = c["B"], c["nodes"], c["hk"], c["page"]
    page = s["table"].long().clamp(min=0)                                  # [B, pages]
    k = _values(s["kc"][page], s["kn"][page], s["tables"])                 # [B, pages, hk, P, d]
    v = _values(s["vc"][page], s["vn"][page], s["tables"])
    k, v = (x.transpose(1, 2).flatten(2, 3) for x in (k, v))               # [B, hk, S, d]
    q = s["q"].float().view(B, n, hk, -1, c["d"]).permute(0, 2, 3, 1, 4).flatten(2, 3)
    x = (q @ k.transpose(-1, -2)).unflatten(2, (-1, n)) * s["scale"]       # [B, hk, G, n, S]
    x = x.masked_fill(~_visible(s, k.shape[2])[:, None, None], -torch.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True))
    o = (x.flatten(2, 3) @ v).unflatten(2, (-1, n)) / x.sum(-1, keepdim=True)
    return o.permute(0, 3, 1, 2, 4).reshape(B * n, c["hq"], c["d"]).to(s["q"].dtype)


def _visible(s, S):
    """[B, nodes, S]: the prefix, and the nodes that a node's mask names (its ancestors)."""
    c = s["case"]
    n = c["nodes"]
    node = torch.arange(S, device="cuda") - s["prefix"][:, None]           # [B, S]
    j = node.clamp(0, n - 1)
    i = torch.arange(n, device="cuda")
    if s["mask"] is None:
        sees = j[:, None, :] <= i[:, None]
    else:
        sees = (s["mask"].view(-1, n, 1) >> j[:, None, :]) & 1 == 1
    return (node < 0)[:, None] | ((node < n)[:, None] & sees)


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return {"q": _rope_exact(s, s["q"]), "k": _rope_exact(s, s["k"])}
    R = _rotation_matrix(s["tables"])
    if case["op"] == "store":
        k, kn = _store_exact(s, s["k"], R)
        v, vn = _store_exact(s, s["v"], R)
        return {"k": k, "v": v, "k_norms": kn, "v_norms": vn}
    return _attend_exact(s, R)


def _rope_exact(s, x):
    """A pair is a complex number, and a position a turn of it."""
    c = s["case"]
    rot, y = c["rot"], x.double().clone()
    turn = torch.polar(torch.full_like(s["freq"], s["amp"]).expand(c["T"], -1).contiguous(),
                       torch.outer(s["pos"].double(), s["freq"]))
    turn = (turn.conj() if c["inverse"] else turn)[:, None]
    first = (slice(0, rot // 2), slice(rot // 2, rot)) if c["layout"] == "half" else (
        slice(0, rot, 2), slice(1, rot, 2))
    z = torch.complex(y[..., first[0]].contiguous(), y[..., first[1]].contiguous()) * turn
    y[..., first[0]], y[..., first[1]] = z.real, z.imag
    return y


def _rotation_matrix(tab):
    """R as a dense matrix: row i has H[i, j] sign[j] / sqrt(h) at column perm[j]."""
    d, h = tab["sign"].numel(), tab["had"].shape[0]
    R = torch.zeros(d, d, dtype=torch.float64, device="cuda")
    blocks = torch.block_diag(*[tab["had"]] * (d // h)) / math.sqrt(h)
    R[:, tab["perm"]] = blocks * tab["sign"]
    return R


def _store_exact(s, x, R):
    c, cent, bound = s["case"], s["tables"]["cent"], s["tables"]["bound"]
    z = x.double() @ R.T
    norm = torch.linalg.vector_norm(z, dim=-1)
    code = torch.searchsorted(bound, (z * (math.sqrt(c["d"]) / (norm + EPS))[..., None]),
                              right=True)
    back = (cent[code] @ R) * (norm / math.sqrt(c["d"]))[..., None]
    kept = s["slots"] >= 0
    back[~kept] = 0
    norms = torch.zeros(s["kn"].shape, dtype=torch.float64, device="cuda")
    slot = s["slots"][kept]
    norms[slot // c["page"], :, slot % c["page"]] = norm[kept]
    return back, norms


def _attend_exact(s, R):
    """One sequence at a time: the visible rows gathered token by token, a softmax over them."""
    c, cent = s["case"], s["tables"]["cent"]
    n, P, d, G = c["nodes"], c["page"], c["d"], c["hq"] // c["hk"]
    out = torch.zeros(c["B"] * n, c["hq"], d, dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        S = int(s["prefix"][b]) + n
        t = torch.arange(S, device="cuda")
        page, at = s["table"][b].long()[t // P], t % P
        q = s["q"][b * n:(b + 1) * n].double()
        see = torch.ones(n, S, dtype=torch.bool, device="cuda")
        see[:, S - n:] = torch.ones(n, n, device="cuda").tril().bool()
        if s["mask"] is not None:
            words = s["mask"][b * n:(b + 1) * n].tolist()
            see[:, S - n:] = torch.tensor([[bool(w >> j & 1) for j in range(n)] for w in words],
                                          device="cuda")
        for g in range(c["hk"]):
            k, v = (cent[_bits(x[page, g, at], c["bits"])] * (m[page, g, at].double()
                    / math.sqrt(d))[:, None] @ R for x, m in ((s["kc"], s["kn"]),
                                                             (s["vc"], s["vn"])))
            score = torch.einsum("ngd,sd->gns", q[:, g * G:(g + 1) * G], k) * s["scale"]
            p = torch.softmax(score.masked_fill(~see, -torch.inf), -1)
            out[b * n:(b + 1) * n, g * G:(g + 1) * G] = torch.einsum("gns,sd->ngd", p, v)
    return out


def _bits(packed, bits):
    """Codes from bytes, bit by bit."""
    bit = (packed[..., None] >> torch.arange(8, device="cuda")) & 1
    bit = bit.flatten(-2).unflatten(-1, (-1, bits)).long()
    return (bit << torch.arange(bits, device="cuda")).sum(-1)
