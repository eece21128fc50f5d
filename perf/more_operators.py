"""The operators of a verification pass whose target keeps one latent vector a
token (latent attention) and draws its tokens at random, and the work they are
measured on.

  append   dt_latent_append     norm of the latents, rotation of the shared key
                                part and of the queries, into a paged cache
  absorb   dt_latent_attention  attention of a chunk of new tokens over the
                                latents themselves (absorbed form)
  prefill  dt_latent_prefill    the same with every head's keys and values made
                                from the latents (expanded form)
  commit   dt_latent_commit     the accepted path of a tree, and its latents
                                moved to the front of the chunk's slots
  sample   dt_sample_rows       a token for every row of logits: temperature,
                                top-k, top-p, min-p, from given random numbers

``own`` chooses between the plain forms (elementary torch operations in 32
bits, 64 for angles, and for the sums that decide which token is drawn) and the
library's kernels.  Lengths of a ragged batch are spread evenly over the case's
range and dealt to the requests by the seed, so that the work of a case is the
same for every seed.
"""

import math

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}

# How requests draw their tokens: temperature, top_k, top_p, min_p (0, 1 and 0: off).
_SETTINGS = [(0.7, 50, 0.95, 0.0),         # the usual chat setting
             (0.0, 0, 1.0, 0.0),           # greedy
             (1.0, 0, 0.9, 0.0),
             (1.0, 0, 1.0, 0.05),
             (1.0, 0, 1.0, 0.0),           # the model's own distribution
             (0.8, 1000, 0.98, 0.01),
             (1.3, 0, 0.99, 0.0),          # wide
             (0.6, 20, 1.0, 0.0)]


def listed():
    return [
        # one request generates one token: latency
        dict(name="append_one_token", op="append", B=1, lead=1, n_max=0, nn_lo=0, ctx_lo=4000, ctx_hi=4000, Hq=16,
             Dc=512, Dr=64, Dn=128, page=16, dtype="bf16", norm=True, interleaved=False),
        # two long prompts, far into their context, all heads of a wide model, pairs of neighbours
        dict(name="append_chunk_far", op="append", B=2, lead=0, n_max=4096, nn_lo=3001, ctx_lo=60001, ctx_hi=100003,
             Hq=128, Dc=512, Dr=64, Dn=128, page=64, dtype="f16", norm=True, interleaved=True),
        # one request generates one token over a long context: latency
        dict(name="absorb_one_token", op="absorb", B=1, lead=1, n_max=0, nn_lo=0, ctx_lo=4095, ctx_hi=4095, Hq=16,
             Dc=512, Dr=64, page=16, dtype="bf16"),
        # a ragged batch generates one token each, heads split over devices: the cache's bandwidth
        dict(name="absorb_decode_b64", op="absorb", B=64, lead=1, n_max=0, nn_lo=0, ctx_lo=33, ctx_hi=16383, Hq=16,
             Dc=512, Dr=64, page=16, dtype="bf16"),
        # the same with all heads on one device: the matrix cores
        dict(name="absorb_decode_heads", op="absorb", B=64, lead=1, n_max=0, nn_lo=0, ctx_lo=33, ctx_hi=16383, Hq=128,
             Dc=512, Dr=64, page=64, dtype="bf16"),
        # trees of the benchmark's budget over long contexts, a smaller latent
        dict(name="absorb_tree_b8", op="absorb", B=8, lead=1, n_max=64, nn_lo=57, ctx_lo=6001, ctx_hi=10007, Hq=28,
             Dc=256, Dr=32, page=32, dtype="f16"),
        # a short prompt
        dict(name="prefill_short", op="prefill", B=1, lead=0, n_max=300, nn_lo=300, ctx_lo=211, ctx_hi=211, Hq=16,
             Dc=512, Dr=64, Dn=128, page=16, dtype="bf16"),
        # a chunk of a long prompt
        dict(name="prefill_chunk", op="prefill", B=2, lead=0, n_max=2048, nn_lo=1801, ctx_lo=6005, ctx_hi=14001, Hq=32,
             Dc=512, Dr=64, Dn=128, page=64, dtype="bf16"),
        # one request commits its path in 16 layers
        dict(name="commit_one", op="commit", B=1, lead=1, n_max=64, nn_lo=64, W=8, ctx_lo=333, ctx_hi=333, layers=16,
             Dc=512, Dr=64, page=16, dtype="bf16", accepted=5),
        # the benchmark's batch
        dict(name="commit_b64", op="commit", B=64, lead=1, n_max=64, nn_lo=57, W=8, ctx_lo=9, ctx_hi=130, layers=32,
             Dc=512, Dr=64, page=16, dtype="bf16", accepted=7),
        # one request's next token
        dict(name="sample_one", op="sample", B=1, lead=1, n_max=0, nn_lo=0, V=32000, dtype="f32", first=0),
        # the target's rows of 64 requests after drafts of seven tokens, each request with a setting of its own
        dict(name="sample_draft_b64", op="sample", B=64, lead=1, n_max=7, nn_lo=7, V=151936, dtype="bf16", first=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    biggest = {}
    for c in listed():
        w = work(c)
        b = biggest.setdefault(c["op"], [0, 0])
        b[0], b[1] = max(b[0], w["bytes"]), max(b[1], w["flops"])
    while True:
        c = _draw_one(rng)
        w = work(c)
        b = biggest[c["op"]]
        if w["bytes"] <= b[0] and w["flops"] <= b[1]:
            return c


def _draw_one(rng):
    op = rng.choice(["append", "absorb", "absorb", "prefill", "commit", "sample"])
    c = dict(op=op)
    kind = dict(append=rng.choice(["one", "tree", "chunk"]), absorb=rng.choice(["one", "one", "tree", "chunk"]),
                prefill=rng.choice(["chunk", "chunk", "tree"]), commit="tree",
                sample=rng.choice(["one", "tree"]))[op]
    if kind == "one":
        c.update(B=_log_int(rng, 1, 64), lead=1, n_max=0, nn_lo=0)
    elif kind == "tree":
        n = _log_int(rng, 5, 256)
        c.update(B=_log_int(rng, 1, 64), lead=rng.choice([1, 1, 1, 2, 3]), n_max=n, nn_lo=rng.randint(n // 2, n))
    else:
        n = _log_int(rng, 17, 4096 if op != "absorb" else 512)
        c.update(B=_log_int(rng, 1, 8), lead=0, n_max=n, nn_lo=rng.randint(n // 2 + 1, n))
    if op == "sample":
        c.update(V=rng.choice([_log_int(rng, 10, 40000), 32000, 151936, rng.randint(100000, 160000)]),
                 dtype=rng.choice(["bf16", "f32"]), first=rng.randint(0, len(_SETTINGS) - 1))
        c["B"] = min(c["B"], max(1, 78000000 // (c["V"] * (c["lead"] + c["n_max"]))))
        return c
    c.update(Dc=rng.choice([256, 512, 512]), Dr=rng.choice([32, 64, 64]),
             page=rng.choice([1, 8, 16, 16, 24, 32, 64, 128, 256]), dtype=rng.choice(["bf16", "f16"]))
    if op == "append":
        hi = _log_int(rng, 300, 100000 // c["B"] + 301)
        c.update(Hq=_log_int(rng, 1, 128), Dn=rng.choice([64, 128]), norm=rng.random() < 0.8,
                 interleaved=rng.random() < 0.5)
    elif op == "absorb":
        hi = _log_int(rng, 40, 16383)
        c.update(Hq=rng.choice([_log_int(rng, 1, 128), 16, 128]))
    elif op == "prefill":
        hi = _log_int(rng, 40, 14001)
        c.update(Hq=_log_int(rng, 1, 32), Dn=rng.choice([64, 128]))
    else:
        hi = _log_int(rng, 20, 200)
        c.update(layers=rng.randint(1, 32), W=_log_int(rng, 2, 16), accepted=rng.randint(1, 7))
    c.update(ctx_lo=rng.randint(hi // 4, hi), ctx_hi=hi)
    return c


# ---------------------------------------------------------------------------
# lengths, trees, caches
# ---------------------------------------------------------------------------

def _spread(lo, hi, n):
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _lengths(case):
    """(ctx_len, n_nodes) of the requests before the seed deals them out; they
    are dealt together."""
    ctx = _spread(case["ctx_lo"], case["ctx_hi"], case["B"]) if "ctx_lo" in case else [0] * case["B"]
    return ctx, _spread(case["nn_lo"], case["n_max"], case["B"])


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    ctx, nn = _lengths(case)
    rows = [case["lead"] + n for n in nn]
    keys = sum(c + r for c, r in zip(ctx, rows))
    pairs = sum(c * r + (r * (r + 1) // 2 if case["lead"] == 0 else r) for c, r in zip(ctx, rows))
    if case["op"] == "append":
        elems = sum(rows) * (case["Dc"] + case["Dr"] * (1 + case["Hq"]))
        return {"bytes": 2 * elems * size, "flops": 10 * elems}
    if case["op"] == "absorb":
        Dc, Dr = case["Dc"], case["Dr"]
        return {"bytes": size * (keys * (Dc + Dr) + sum(rows) * case["Hq"] * (2 * Dc + Dr)),
                "flops": 2 * pairs * case["Hq"] * (2 * Dc + Dr)}
    if case["op"] == "prefill":
        Dc, Dr, Dn, Hq = case["Dc"], case["Dr"], case["Dn"], case["Hq"]
        return {"bytes": size * (keys * (Dc + Dr) + 2 * Hq * Dn * Dc + sum(rows) * Hq * (2 * Dn + Dr)),
                "flops": 2 * pairs * Hq * (2 * Dn + Dr) + 4 * keys * Hq * Dn * Dc}
    if case["op"] == "sample":
        elems = sum(rows) * case["V"]
        return {"bytes": elems * size + 12 * sum(rows), "flops": 8 * elems}
    moved = case["B"] * case["accepted"] * case["layers"] * (case["Dc"] + case["Dr"])
    return {"bytes": 2 * moved * size + 16 * sum(rows), "flops": sum(rows)}


def _deal(case, gen):
    order = torch.randperm(case["B"], generator=gen)
    ctx, nn = _lengths(case)
    return torch.tensor(ctx)[order].tolist(), torch.tensor(nn)[order].tolist()


def _trees(rs, nn, n_max, W):
    """Trees in BFS order, W nodes to a depth: parents, depths and the packed
    ancestor masks (reflexive, lowest node in the lowest bit)."""
    B, words = len(nn), (n_max + 31) // 32
    parents = np.full((B, n_max), -1, np.int32)
    depths = np.zeros((B, n_max), np.int32)
    seen = np.zeros((B, n_max, words * 32), bool)
    for b in range(B):
        for i in range(nn[b]):
            t = i // W
            depths[b, i] = t + 1
            if t > 0:
                parents[b, i] = (t - 1) * W + rs.randint(W)
                seen[b, i] = seen[b, parents[b, i]]
            seen[b, i, i] = True
    mask = np.packbits(seen, axis=-1, bitorder="little").view(np.int32)
    return parents, depths, mask


def _cache(case, ctx, rs, gpu, layers=1):
    """A cache whose pages are dealt out in random order, filled with earlier
    latents and keys' rotated parts."""
    P, rows = case["page"], case["lead"] + case["n_max"]
    need = [(c + rows + P - 1) // P for c in ctx]
    total, width = sum(need), max(need)
    order = rs.permutation(total).astype(np.int32)
    table = np.full((len(ctx), width), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    c = torch.empty(layers, total, P, case["Dc"] + case["Dr"], dtype=_TYPES[case["dtype"]], device="cuda")
    c.normal_(generator=gpu)
    return c, torch.from_numpy(table).cuda()


def _frequencies(case):
    """Radians a position, in 64 bits: base 1e4."""
    return 1e4 ** (-np.arange(0, case["Dr"], 2, dtype=np.float64) / case["Dr"])


def _scale(case):
    """Scores are those of heads with Dn unrotated and Dr rotated elements."""
    return (case.get("Dn", 128) + case["Dr"]) ** -0.5


def prepare(case, seed):
    gen = torch.Generator().manual_seed(seed * 7919 + 17)
    gpu = torch.Generator(device="cuda").manual_seed(seed * 104729 + 3)
    rs = np.random.RandomState((seed * 65537 + 11) % (1 << 32))
    ctx, nn = _deal(case, gen)
    B, lead, n_max = case["B"], case["lead"], case["n_max"]
    rows = lead + n_max
    t = _TYPES[case["dtype"]]

    def ints(x):
        return torch.tensor(x, dtype=torch.int32).cuda()

    def normal(*shape, dtype=t, sd=1.0):
        return torch.empty(*shape, dtype=torch.float32, device="cuda").normal_(generator=gpu).mul_(sd).to(dtype)

    s = dict(case=case, n_nodes=ints(nn), nn=nn, ctx=ctx)
    if case["op"] == "sample":
        return _prepare_sample(case, s, rs, normal)
    if lead > 0 and n_max > 0:
        parents, depths, mask = _trees(rs, nn, n_max, case.get("W", 16 if n_max > 128 else 8))
        s.update(parents=torch.from_numpy(parents).cuda(), depths=torch.from_numpy(depths).cuda(),
                 mask=torch.from_numpy(mask).cuda())
    else:
        s.update(parents=None, depths=None, mask=None)
    s["ctx_len"] = ints(ctx)
    s["c"], s["table"] = _cache(case, ctx, rs, gpu, case.get("layers", 1))
    Dc, Dr, Hq, Dn = case["Dc"], case["Dr"], case.get("Hq"), case.get("Dn")
    if case["op"] == "append":
        # two projections' outputs: latent and shared key part side by side, and the queries' heads, of whose
        # Dn + Dr elements the last Dr are rotated; they go behind the Dc elements that the absorbed product makes
        down = normal(B, rows, Dc + Dr)
        q = normal(B, rows, Hq, Dn + Dr)
        q_full = torch.zeros(B, rows, Hq, Dc + Dr, dtype=t, device="cuda")
        s.update(latent=down[..., :Dc], k_rot=down[..., Dc:], q_rot=q[..., Dn:], q_out=q_full[..., Dc:], norm=None,
                 freqs=torch.from_numpy(_frequencies(case)).cuda())
        if case["norm"]:
            s["norm"] = (normal(Dc, dtype=torch.float32, sd=0.2) + 1).to(t)
    elif case["op"] == "absorb":
        # absorbed queries: their scores over the Dc elements have the spread that Dn elements give
        q = normal(B, rows, Hq, Dc + Dr, dtype=torch.float32)
        q[..., :Dc] *= math.sqrt(128 / Dc)
        q = q.to(t)
        s.update(q=q, out=torch.zeros(B, rows, Hq, Dc, dtype=t, device="cuda"), keys=max(ctx) + rows)
    elif case["op"] == "prefill":
        s.update(q=normal(B, rows, Hq, Dn + Dr), weight=normal(Hq, 2 * Dn, Dc, sd=Dc ** -0.5),
                 out=torch.zeros(B, rows, Hq, Dn, dtype=t, device="cuda"), keys=max(ctx) + rows)
    else:
        V, stop = 151936, 151935
        tokens = rs.randint(0, stop, (B, n_max)).astype(np.int32)
        target = np.full((B, rows), stop, np.int32)
        host = s["parents"].cpu().numpy()
        depth = s["depths"].cpu().numpy()
        for b in range(B):
            # a path of the wanted length whose nodes all lie behind the slots it moves to
            for a in range(case["accepted"], 0, -1):
                paths = []
                for leaf in np.flatnonzero(depth[b, :nn[b]] == a):
                    path = [int(leaf)]
                    while host[b, path[0]] >= 0:
                        path.insert(0, int(host[b, path[0]]))
                    if path[0] >= a:
                        paths.append(path)
                if paths:
                    cur = -1
                    for node in paths[rs.randint(len(paths))]:
                        target[b, lead + cur] = tokens[b, node]
                        cur = node
                    break
        L = n_max + 1
        s.update(tokens=torch.from_numpy(tokens).cuda(), target=torch.from_numpy(target).cuda(),
                 steps=min(int(depth.max()) + 1, L), accepted=torch.zeros(B, L, dtype=torch.int32, device="cuda"),
                 lengths=torch.zeros(B, dtype=torch.int32, device="cuda"),
                 nodes=torch.zeros(B, L, dtype=torch.int32, device="cuda"))
    if own:
        from draft_tree_construction_dt_amd import binding as bd
        s["cache"] = bd.LatentCache(s["c"], s["table"], Dr)
        s["chunk"] = bd.Chunk(ctx_len=s["ctx_len"], lead=lead, n_max=n_max, n_nodes=s["n_nodes"], mask=s["mask"],
                              depths=s["depths"])
        need = 0
        if case["op"] == "absorb":
            need = bd.dt_latent_workspace(s["cache"], s["chunk"], Hq)
        elif case["op"] == "prefill":
            need = bd.dt_latent_prefill_workspace(s["cache"], s["chunk"], Hq, Dn, s["keys"])
        s["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    return s


def _prepare_sample(case, s, rs, normal):
    """Logits of three kinds of rows: a few tokens far above the rest (a model
    that knows what comes next), a broad head, and no head at all; every fifth
    row is under a grammar that forbids half of the tokens."""
    B, V, rows = case["B"], case["V"], case["lead"] + case["n_max"]
    x = normal(B * rows, V, dtype=torch.float32, sd=2.0)
    kind = torch.from_numpy(np.arange(B * rows) % 4).cuda()
    head = min(V, 64)
    ids = torch.from_numpy(rs.randint(0, V, (B * rows, head))).cuda()
    lift = torch.from_numpy(rs.exponential(2.0, (B * rows, head)).astype(np.float32)).cuda()
    lift = lift + torch.where(kind <= 1, 9.0, 6.0)[:, None]
    x.scatter_add_(1, ids, torch.where((kind == 3)[:, None], 0.0, lift))
    barred = torch.from_numpy(rs.rand(V) < 0.5).cuda()
    grammar = torch.from_numpy(np.arange(B * rows) % 5 == 4).cuda()
    x.masked_fill_(grammar[:, None] & barred, float("-inf"))
    x = x.view(B, rows, V).to(_TYPES[case["dtype"]])
    how = [_SETTINGS[(case["first"] + i) % len(_SETTINGS)] for i in rs.permutation(B)]
    temperature, top_k, top_p, min_p = zip(*how)

    def floats(v):
        return torch.tensor(v, dtype=torch.float32).cuda()

    s.update(logits=x, u=torch.from_numpy(rs.rand(B, rows).astype(np.float32).clip(max=1 - 2.0 ** -24)).cuda(),
             temperature=floats(temperature), top_k=torch.tensor(top_k, dtype=torch.int32).cuda(),
             top_p=floats(top_p), min_p=floats(min_p), tokens=torch.zeros(B, rows, dtype=torch.int32, device="cuda"),
             logp=torch.zeros(B, rows, dtype=torch.float32, device="cuda"))
    if own:
        from draft_tree_construction_dt_amd import binding as bd
        need = bd.dt_sample_workspace(x)
        s["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return globals()[("_own_" if own else "_plain_") + s["case"]["op"]](s)


def _own_append(s):
    from draft_tree_construction_dt_amd import binding as bd
    bd.dt_latent_append(s["cache"], s["chunk"], s["latent"], s["k_rot"], q_rot=s["q_rot"], q_out=s["q_out"],
                        norm=s["norm"], eps=1e-6, freqs=s["freqs"], interleaved=s["case"]["interleaved"])
    return s["q_out"], s["c"]


def _own_absorb(s):
    from draft_tree_construction_dt_amd import binding as bd
    bd.dt_latent_attention(s["cache"], s["chunk"], s["q"], s["out"], _scale(s["case"]), workspace=s["workspace"])
    return s["out"]


def _own_prefill(s):
    from draft_tree_construction_dt_amd import binding as bd
    bd.dt_latent_prefill(s["cache"], s["chunk"], s["q"], s["weight"], s["out"], _scale(s["case"]), s["keys"],
                         workspace=s["workspace"])
    return s["out"]


def _own_commit(s):
    from draft_tree_construction_dt_amd import binding as bd
    bd.dt_latent_commit(s["cache"], s["chunk"], s["tokens"], s["parents"], s["target"], s["accepted"], s["lengths"],
                        nodes=s["nodes"])
    return s["accepted"], s["lengths"], s["nodes"], s["c"]


def _own_sample(s):
    from draft_tree_construction_dt_amd import binding as bd
    bd.dt_sample_rows(s["logits"], s["u"], s["tokens"], temperature=s["temperature"], top_k=s["top_k"],
                      top_p=s["top_p"], min_p=s["min_p"], logp=s["logp"], lead=s["case"]["lead"],
                      n_nodes=s["n_nodes"], workspace=s["workspace"])
    return s["tokens"], s["logp"]


def _rows(s):
    """[rows] row numbers, [B][rows] whether a row is one of the request's."""
    c = s["case"]
    r = torch.arange(c["lead"] + c["n_max"], device="cuda")
    return r, r[None] < (c["lead"] + s["n_nodes"])[:, None]


def _slots(s, at):
    """Page and offset of the requests' slots at [B][n]."""
    P = s["case"]["page"]
    return torch.gather(s["table"].long(), 1, at // P), at % P


def _rotate(x, cos, sin, interleaved):
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat((a * cos - b * sin, a * sin + b * cos), -1)


def _plain_append(s):
    c = s["case"]
    r, valid = _rows(s)
    at = s["ctx_len"].long()[:, None] + r
    pos = at
    if s["depths"] is not None:
        nodes = s["ctx_len"].long()[:, None] + c["lead"] - 1 + s["depths"].long()
        pos = torch.cat((at[:, :c["lead"]], nodes), 1)
    angle = pos[:, :, None].double() * s["freqs"]
    cos, sin = angle.cos().float(), angle.sin().float()
    x = s["latent"].float()
    if s["norm"] is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * s["norm"].float()
    x = torch.cat((x, _rotate(s["k_rot"].float(), cos, sin, c["interleaved"])), -1).to(s["c"].dtype)
    q = _rotate(s["q_rot"].float(), cos[:, :, None], sin[:, :, None], c["interleaved"]).to(x.dtype)
    s["q_out"].copy_(torch.where(valid[:, :, None, None], q, s["q_out"]))
    page, off = _slots(s, at)
    cache = s["c"][0]
    cache[page, off] = torch.where(valid[:, :, None], x, cache[page, off])
    return s["q_out"], s["c"]


def _bits(words, n):
    shift = torch.arange(32, device="cuda", dtype=torch.int32)
    return ((words[..., None] >> shift) & 1).flatten(-2)[..., :n].bool()


def _seen(s):
    """[B][rows][keys]: the slots that each row sees."""
    c = s["case"]
    r, _ = _rows(s)
    S, lead = s["keys"], c["lead"]
    rel = torch.arange(S, device="cuda") - s["ctx_len"].long()[:, None]     # a key's row in the chunk, < 0: context
    see = rel[:, None, :] <= r[None, :, None]
    if s["mask"] is not None:
        bits = _bits(s["mask"], c["n_max"])                                 # [B][node][node]
        node = (rel - lead).clamp(0, c["n_max"] - 1)
        marked = torch.gather(bits, 2, node[:, None, :].expand(c["B"], c["n_max"], S)) & (rel >= lead)[:, None]
        marked &= (rel - lead < s["n_nodes"][:, None])[:, None]
        see = torch.cat((see[:, :lead], marked | (rel < lead)[:, None]), 1)
    return see


def _latents(s):
    """[B][keys][Dc + Dr] of the cache, in 32 bits."""
    last = s["ctx_len"].long()[:, None] + s["case"]["lead"] + s["case"]["n_max"] - 1
    at = torch.arange(s["keys"], device="cuda")[None]
    page, off = _slots(s, torch.minimum(at, last))
    return s["c"][0][page, off].float()


def _weights(x, see):
    """Softmax of scores over the keys that are seen; nothing seen: zeros."""
    x = torch.where(see, x, float("-inf"))
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(top == float("-inf"), 0.0, top))
    total = x.sum(-1, keepdim=True)
    return x / torch.where(total == 0, 1.0, total)


def _plain_absorb(s):
    c = s["case"]
    B, R, Hq, Dc = c["B"], c["lead"] + c["n_max"], c["Hq"], c["Dc"]
    k = _latents(s)
    q = s["q"].float().reshape(B, R * Hq, -1)
    x = torch.matmul(q, k.transpose(1, 2).contiguous()).view(B, R, Hq, -1) * _scale(c)
    p = _weights(x, _seen(s)[:, :, None])
    o = torch.matmul(p.view(B, R * Hq, -1), k[..., :Dc].contiguous()).view(B, R, Hq, Dc).to(s["out"].dtype)
    s["out"].copy_(torch.where(_rows(s)[1][:, :, None, None], o, s["out"]))
    return s["out"]


def _plain_prefill(s):
    c = s["case"]
    B, R, Hq, Dc, Dn, Dr = c["B"], c["lead"] + c["n_max"], c["Hq"], c["Dc"], c["Dn"], c["Dr"]
    x = _latents(s)
    kv = torch.matmul(x[..., :Dc], s["weight"].float().view(-1, Dc).T).view(B, -1, Hq, 2 * Dn)
    k = torch.cat((kv[..., :Dn], x[:, :, None, Dc:].expand(-1, -1, Hq, -1)), -1).permute(0, 2, 3, 1).contiguous()
    v = kv[..., Dn:].transpose(1, 2).contiguous()
    y = torch.matmul(s["q"].float().transpose(1, 2).contiguous(), k) * _scale(c)      # [B][Hq][R][keys]
    o = torch.matmul(_weights(y, _seen(s)[:, None]), v).transpose(1, 2).to(s["out"].dtype)
    s["out"].copy_(torch.where(_rows(s)[1][:, :, None, None], o, s["out"]))
    return s["out"]


def _plain_commit(s):
    c = s["case"]
    B, lead, n_max = c["B"], c["lead"], c["n_max"]
    L = s["accepted"].shape[1]
    i = torch.arange(n_max, device="cuda")
    cur = torch.full((B,), -1, device="cuda")
    alive = torch.ones(B, dtype=torch.bool, device="cuda")
    count = torch.zeros(B, dtype=torch.long, device="cuda")
    tokens = torch.full((B, L), -1, dtype=torch.int32, device="cuda")
    nodes = torch.full((B, L), -1, dtype=torch.int32, device="cuda")
    for step in range(s["steps"]):
        want = torch.gather(s["target"], 1, (lead + cur)[:, None])
        fits = (s["parents"] == cur[:, None]) & (s["tokens"] == want) & (i < s["n_nodes"][:, None])
        child = torch.where(fits, i, n_max).amin(1)
        found = alive & (child < n_max) & (step < L - 1)
        tokens[:, step] = torch.where(alive, want[:, 0], -1)
        nodes[:, step] = torch.where(found, child, -1).int()
        count += alive
        cur = torch.where(found, child, cur)
        alive = found
    s["accepted"].copy_(tokens)
    s["lengths"].copy_(count)
    s["nodes"].copy_(nodes)
    n = min(s["steps"], L)
    first = s["ctx_len"].long()[:, None] + lead
    to = first + torch.arange(n, device="cuda")
    source = torch.where(nodes[:, :n] >= 0, first + nodes[:, :n], to)
    last = first + n_max - 1
    (p0, o0), (p1, o1) = _slots(s, torch.minimum(source, last)), _slots(s, torch.minimum(to, last))
    keep = (nodes[:, :n] >= 0)[None, :, :, None]
    cache = s["c"]
    cache[:, p1, o1] = torch.where(keep, cache[:, p0, o0], cache[:, p1, o1])
    return s["accepted"], s["lengths"], s["nodes"], s["c"]


def _plain_sample(s):
    c = s["case"]
    B, V, rows = c["B"], c["V"], c["lead"] + c["n_max"]
    valid = _rows(s)[1]
    x = s["logits"].view(B * rows, V)

    def each(t):
        return t.double()[:, None].expand(B, rows).reshape(-1, 1)

    par = [each(s[n]) for n in ("temperature", "top_k", "top_p", "min_p")]
    u = s["u"].double().view(-1, 1)
    step = max(1, (1 << 26) // V)                                # rows at a time
    tokens, logp = [], []
    for at in range(0, B * rows, step):
        heat, top_k, top_p, min_p = (p[at:at + step] for p in par)
        y, order = torch.sort(x[at:at + step].double(), dim=1, descending=True, stable=True)
        top = y[:, :1]
        empty = top == float("-inf")
        rank = torch.arange(V, device="cuda")
        w = torch.exp((y - torch.where(empty, 0.0, top)) / torch.where(heat > 0, heat, 1.0))
        w = torch.where(heat > 0, w, (rank == 0).double())
        w = torch.where((top_k > 0) & (rank >= top_k), 0.0, w)
        upto = torch.cumsum(w, 1)
        before = torch.cat((torch.zeros_like(upto[:, :1]), upto[:, :-1]), 1)
        keep = (before < top_p * upto[:, -1:]) & (w >= min_p)
        keep[:, 0] = True
        w = torch.zeros_like(w).scatter_(1, order, torch.where(keep, w, 0.0))     # by token again
        upto = torch.cumsum(w, 1)
        token = (upto <= u[at:at + step] * upto[:, -1:]).sum(1, keepdim=True).clamp(max=V - 1)
        chance = torch.log(torch.gather(w, 1, token) / upto[:, -1:])
        tokens.append(torch.where(empty, -1, token))
        logp.append(torch.where(empty, float("-inf"), chance))
    s["tokens"].copy_(torch.where(valid, torch.cat(tokens).view(B, rows).int(), s["tokens"]))
    s["logp"].copy_(torch.where(valid, torch.cat(logp).view(B, rows).float(), s["logp"]))
    return s["tokens"], s["logp"]


# ---------------------------------------------------------------------------
# the definitions in 64 bits, one request at a time
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return globals()["_exact_" + case["op"]](case, s)


def _exact_append(c, s):
    cache, q_out = s["c"].double(), s["q_out"].double()
    f = torch.from_numpy(_frequencies(c)).cuda()
    half = c["Dr"] // 2
    lo = torch.arange(half, device="cuda") * (2 if c["interleaved"] else 1)
    hi = lo + (1 if c["interleaved"] else half)
    table = s["table"].cpu().numpy()
    depths = None if s["depths"] is None else s["depths"].cpu().numpy()

    def turned(x, z):
        y = x.double().clone()
        w = torch.complex(y[..., lo], y[..., hi]) * z
        y[..., lo], y[..., hi] = w.real, w.imag
        return y

    for b in range(c["B"]):
        n = c["lead"] + s["nn"][b]
        pos = [s["ctx"][b] + r for r in range(n)]
        if depths is not None:
            pos[c["lead"]:] = [s["ctx"][b] + c["lead"] - 1 + int(depths[b, i]) for i in range(s["nn"][b])]
        angle = torch.tensor(pos, dtype=torch.float64).cuda()[:, None] * f
        z = torch.polar(torch.ones_like(angle), angle)
        slot = s["ctx"][b] + np.arange(n)
        page = torch.from_numpy(table[b][slot // c["page"]].astype(np.int64)).cuda()
        off = torch.from_numpy(slot % c["page"]).cuda()
        x = s["latent"][b, :n].double()
        if s["norm"] is not None:
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / c["Dc"] + 1e-6) * s["norm"].double()
        cache[0, page, off] = torch.cat((x, turned(s["k_rot"][b, :n], z)), -1)
        q_out[b, :n] = turned(s["q_rot"][b, :n], z[:, None])
    return q_out, cache


def _request(c, s, b, table):
    """(rows, latents of the request's keys in 64 bits, what its rows see)."""
    nn, ctx, lead = s["nn"][b], s["ctx"][b], c["lead"]
    rows = lead + nn
    slot = np.arange(ctx + rows)
    flat = torch.from_numpy(table[b][slot // c["page"]].astype(np.int64) * c["page"] + slot % c["page"]).cuda()
    see = torch.ones(rows, rows, dtype=torch.bool, device="cuda").tril()
    if s["mask"] is not None:
        words = s["mask"][b].cpu().numpy().view(np.uint32)[:nn]
        bits = np.unpackbits(words.view(np.uint8), axis=1, bitorder="little")[:, :nn].astype(bool)
        see[lead:, :lead] = True
        see[lead:, lead:] = torch.from_numpy(bits).cuda()
    return rows, s["c"][0].flatten(0, 1)[flat].double(), see


def _exact_absorb(c, s):
    out = s["out"].double()
    table = s["table"].cpu().numpy()
    for b in range(c["B"]):
        rows, x, see = _request(c, s, b, table)
        for r0 in range(0, rows, 64):
            n = min(64, rows - r0)
            q = s["q"][b, r0:r0 + n].double().flatten(0, 1)
            y = (q @ x.T).div_(math.sqrt(128 + c["Dr"])).view(n, c["Hq"], -1)
            y[:, :, s["ctx"][b]:].masked_fill_(~see[r0:r0 + n, None], float("-inf"))
            out[b, r0:r0 + n] = torch.softmax(y, -1) @ x[:, :c["Dc"]]
    return out


def _exact_prefill(c, s):
    out = s["out"].double()
    table = s["table"].cpu().numpy()
    for b in range(c["B"]):
        rows, x, see = _request(c, s, b, table)
        for h in range(c["Hq"]):
            w = s["weight"][h].double()
            k, v = x[:, :c["Dc"]] @ w[:c["Dn"]].T, x[:, :c["Dc"]] @ w[c["Dn"]:].T
            q = s["q"][b, :rows, h].double()
            y = (q[:, :c["Dn"]] @ k.T + q[:, c["Dn"]:] @ x[:, c["Dc"]:].T) / math.sqrt(c["Dn"] + c["Dr"])
            y[:, s["ctx"][b]:].masked_fill_(~see, float("-inf"))
            out[b, :rows, h] = torch.softmax(y, -1) @ v
    return out


def _exact_commit(c, s):
    cache = s["c"].double()
    L = s["accepted"].shape[1]
    accepted, nodes, lengths = [], [], []
    tokens, parents, target, table = (s[n].cpu().tolist() for n in ("tokens", "parents", "target", "table"))
    for b in range(c["B"]):
        cur, path, said = -1, [], []
        while True:
            want = target[b][c["lead"] + cur]
            said.append(want)
            child = [i for i in range(s["nn"][b]) if parents[b][i] == cur and tokens[b][i] == want]
            if not child or len(path) == L - 1:
                break
            cur = child[0]
            path.append(cur)
        accepted.append(said + [-1] * (L - len(said)))
        nodes.append(path + [-1] * (L - len(path)))
        lengths.append(len(said))
        first = s["ctx"][b] + c["lead"]
        old = [cache[:, table[b][(first + n) // c["page"]], (first + n) % c["page"]].clone() for n in path]
        for i, x in enumerate(old):
            cache[:, table[b][(first + i) // c["page"]], (first + i) % c["page"]] = x
    as_int = dict(dtype=torch.int32, device="cuda")
    return (torch.tensor(accepted, **as_int), torch.tensor(lengths, **as_int), torch.tensor(nodes, **as_int), cache)


def _exact_sample(c, s):
    if c["B"] * (c["lead"] + c["n_max"]) * c["V"] > 80000000:
        return None
    V = c["V"]
    tokens, logp = s["tokens"].cpu().numpy().copy(), s["logp"].double().cpu().numpy()
    host = {n: s[n].cpu().numpy() for n in ("temperature", "top_k", "top_p", "min_p", "u")}
    for b in range(c["B"]):
        heat, k, p, low = (float(host[n][b]) for n in ("temperature", "top_k", "top_p", "min_p"))
        for r in range(c["lead"] + s["nn"][b]):
            x = s["logits"][b, r].double().cpu().numpy()
            best = int(np.argmax(x))
            if x[best] == -np.inf:
                tokens[b, r], logp[b, r] = -1, -np.inf
                continue
            if heat <= 0:
                tokens[b, r], logp[b, r] = best, 0.0
                continue
            order = np.argsort(-x, kind="stable")
            if 0 < k < V:
                order = order[:int(k)]
            w = np.exp((x[order] - x[best]) / heat)
            n = 1 + int(np.sum(np.cumsum(w)[:-1] < p * math.fsum(w))) if p < 1 else len(w)
            n = max(1, min(n, int(np.sum(w >= low))))
            kept = np.sort(order[:n])
            w = np.exp((x[kept] - x[best]) / heat)
            upto = np.cumsum(w)
            i = int(np.searchsorted(upto, float(host["u"][b, r]) * upto[-1], side="right"))
            tokens[b, r], logp[b, r] = kept[i], math.log(w[i] / upto[-1])
    return torch.from_numpy(tokens).cuda(), torch.from_numpy(logp).cuda()
