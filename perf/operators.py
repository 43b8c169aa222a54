"""What the tree-decoding operators are measured on.

A hybrid decoder verifies a tree of drafted tokens in one step: every node sees the committed
prefix and its own ancestors.  Five operators make that step and its commit:

  rope      gdn_qk_norm_rope        RMS norm of q and k per head and rotary positions, k and v into cache rows
  attention gdn_attention_tree      softmax attention of the nodes over the cache and their ancestors, gated
  delta     gdn_decode_tree         the gated delta rule's outputs of the nodes, the state left as it was
  commit    gdn_decode_tree_commit  the state advanced along the accepted path
  append    gdn_attn_tree_commit    the accepted nodes' keys and values appended to the cache

A tree is parent[n][t]: -1 a child of the committed prefix, 0 .. t - 1 an earlier node, -2 no node (the
padding of a batch whose trees have fewer nodes).  `accepted[n]` is the last node of the accepted path or -1.
"""
import math

import torch

own = False

EPS = 1e-6
BF16 = torch.bfloat16


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the verification of one 21-node tree: 24 query and 4 key heads of 256, the first 64 dims turned
        {"name": "rope-tree-21", "op": "rope", "tokens": 21, "heads": 24, "kv_heads": 4, "dim": 256, "rotary": 64,
         "interleaved": False, "scaling": "none", "base": 1e7, "factor": 1.0, "far": 262144},
        # a long prompt's keys and queries: whole heads of 128, interleaved pairs, frequencies stretched eight-fold
        {"name": "rope-prompt-32k", "op": "rope", "tokens": 32768, "heads": 32, "kv_heads": 8, "dim": 128, "rotary": 128,
         "interleaved": True, "scaling": "yarn", "base": 1e6, "factor": 8.0, "far": 262144},
        # one new token of one short sequence: the latency of a call
        {"name": "attention-one-777", "op": "attention", "seqs": 1, "nodes": 1, "ctx": 777, "heads": 24, "kv_heads": 4,
         "dim": 256, "ragged": False, "shape": "chain", "gate": True},
        # a serving batch of ragged contexts, 16-node trees
        {"name": "attention-batch-64x16", "op": "attention", "seqs": 64, "nodes": 16, "ctx": 8192, "heads": 24,
         "kv_heads": 4, "dim": 256, "ragged": True, "shape": "bushy", "gate": True},
        # one sequence at the full context with the largest tree
        {"name": "attention-full-262144x64", "op": "attention", "seqs": 1, "nodes": 64, "ctx": 262144, "heads": 24,
         "kv_heads": 4, "dim": 256, "ragged": False, "shape": "bushy", "gate": True},
        # one sequence, 13 nodes: the latency of a delta-rule layer's verification
        {"name": "delta-one-13", "op": "delta", "seqs": 1, "nodes": 13, "key_heads": 16, "value_heads": 48, "shape": "bushy"},
        # the decode batch with small trees: the states' bytes dominate
        {"name": "delta-batch-256x8", "op": "delta", "seqs": 256, "nodes": 8, "key_heads": 16, "value_heads": 48,
         "shape": "bushy"},
        # large trees for a middling batch: the products dominate
        {"name": "delta-batch-64x61", "op": "delta", "seqs": 64, "nodes": 61, "key_heads": 16, "value_heads": 48,
         "shape": "bushy"},
        # the accepted path of one sequence's tree
        {"name": "commit-one-16", "op": "commit", "seqs": 1, "nodes": 16, "key_heads": 16, "value_heads": 48, "shape": "bushy"},
        # and of the decode batch
        {"name": "commit-batch-256x8", "op": "commit", "seqs": 256, "nodes": 8, "key_heads": 16, "value_heads": 48,
         "shape": "chain"},
        # the accepted rows of a few sequences, of another cache's heads
        {"name": "append-5x31", "op": "append", "seqs": 5, "nodes": 31, "kv_heads": 8, "dim": 128, "shape": "chain"},
        # the accepted rows of a full batch with long drafts
        {"name": "append-256x64", "op": "append", "seqs": 256, "nodes": 64, "kv_heads": 4, "dim": 256, "shape": "chain"},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "attention", "attention", "delta", "delta", "commit", "append"])
    shape = rng.choice(["bushy", "bushy", "chain"])
    if op == "rope":
        dim = rng.choice([64, 128, 256])
        kv = rng.choice([1, 2, 4, 8])
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        return {"op": op, "tokens": _spread(rng, 1, 24000), "heads": kv * rng.choice([1, 4, 6]), "kv_heads": kv, "dim": dim,
                "rotary": rng.choice([dim // 4, dim // 2, dim]), "interleaved": rng.random() < 0.5, "scaling": scaling,
                "base": rng.choice([1e4, 1e6, 1e7]), "factor": 1.0 if scaling == "none" else float(rng.choice([2, 4, 8])),
                "far": _spread(rng, 1000, 1000000)}
    if op == "attention":
        dim = rng.choice([128, 256])
        kv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 3, 4, 6, 8])
        seqs, nodes = _spread(rng, 1, 96), _spread(rng, 1, 64)
        # tokens of all contexts such that neither the caches nor the plain form's scores pass the listed cases'
        most = min(64 * 8192 * 4 * 256 // (kv * dim), 64 * 262144 * 24 // (nodes * kv * group)) // seqs
        return {"op": op, "seqs": seqs, "nodes": nodes, "ctx": _spread(rng, 1, max(1, min(262144, most))),
                "heads": kv * group, "kv_heads": kv, "dim": dim, "ragged": rng.random() < 0.6, "shape": shape,
                "gate": rng.random() < 0.6}
    if op in ("delta", "commit"):
        kh, group = rng.choice([2, 4, 8, 16]), rng.choice([1, 2, 3, 4])
        nodes = _spread(rng, 1, 64)
        most = min(256 * 48 // (kh * group), 64 * 61 * 48 // (nodes * kh * group))
        return {"op": op, "seqs": _spread(rng, 1, max(1, min(256, most))), "nodes": nodes, "key_heads": kh,
                "value_heads": kh * group, "shape": shape}
    return {"op": op, "seqs": _spread(rng, 1, 256), "nodes": _spread(rng, 1, 64), "kv_heads": rng.choice([1, 2, 4]),
            "dim": rng.choice([128, 256]), "shape": shape}


def _lengths(case):
    """The contexts: all of the same length, or from an eighth of it to all of it, in an order that is not sorted."""
    n, ctx = case["seqs"], case["ctx"]
    if not case["ragged"] or n == 1:
        return [ctx] * n
    low = max(1, ctx // 8)
    return [low + (ctx - low) * ((i * 7) % n) // (n - 1) if n % 7 else low + (ctx - low) * i // (n - 1) for i in range(n)]


def _live(case):
    """How many of each sequence's T nodes there are: a batch of several pads every third tree."""
    t = case["nodes"]
    return [max(1, t - t // 4) if n % 3 == 1 else t for n in range(case["seqs"])]


def _accepted_nodes(case):
    """The length of each accepted path at most: the first drafted tokens of a run, none for every seventh sequence."""
    return [0 if n % 7 == 6 else min(_live(case)[n], 1 + (n * 5) % 8) for n in range(case["seqs"])]


# ------------------------------------------------------------------ inputs

def _tree(case, gen):
    """parent int32 [N][T] and accepted int32 [N] on the GPU."""
    n, t = case["seqs"], case["nodes"]
    step = torch.arange(t, device="cuda")
    if case["shape"] == "chain":
        parent = (step - 1).expand(n, t).clone()
    else:  # a run of the likeliest tokens first, then branches anywhere
        anywhere = (torch.rand(n, t, generator=gen, device="cuda") * (step + 1)).long().clamp(max=t) - 1
        anywhere = torch.minimum(anywhere, step - 1)
        parent = torch.where(step < min(t, 8), step - 1, anywhere)
    live = torch.tensor(_live(case), device="cuda")
    parent = torch.where(step < live[:, None], parent, torch.full_like(parent, -2))
    accepted = torch.tensor(_accepted_nodes(case), device="cuda") - 1  # the first nodes are a run in both shapes
    return parent.to(torch.int32).contiguous(), accepted.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=BF16):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    op, s = case["op"], {"case": case}
    if op == "rope":
        n, h, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        # q, k and v are columns of one projection, as the layer's input product leaves them
        proj = normal(n, (h + 2 * hk) * d, std=2.0)
        s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, d)) for x in proj.split([h * d, hk * d, hk * d], 1))
        s["q_w"], s["k_w"] = (1 + normal(d, std=0.1, dtype=torch.float32)).to(BF16), (1 + normal(d, std=0.1, dtype=torch.float32)).to(BF16)
        s["positions"] = torch.randint(0, case["far"], (n,), generator=gen, device="cuda", dtype=torch.int32)
        # the cache rows are some of a few more, in no order
        s["n_rows"] = n + n // 16 + 3
        s["rows"] = torch.randperm(s["n_rows"], generator=gen, device="cuda")[:n].contiguous()
        s["k_out"] = torch.zeros(s["n_rows"], hk, d, dtype=BF16, device="cuda")
        s["v_out"] = torch.zeros(s["n_rows"], hk, d, dtype=BF16, device="cuda")
        return s
    s["parent"], s["accepted"] = _tree(case, gen)
    n, t = case["seqs"], case["nodes"]
    if op == "attention":
        h, hk, d = case["heads"], case["kv_heads"], case["dim"]
        lens = _lengths(case)
        cap = max(lens) + 64
        s["len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["q"] = normal(n * t, h, d)
        # keys and values of the nodes and the gate are read where the projection has them
        proj = normal(n * t, (h + 2 * hk) * d)
        s["g"] = proj[:, :h * d].unflatten(1, (h, d)) if case["gate"] else None
        s["k_tree"], s["v_tree"] = proj[:, h * d:(h + hk) * d].unflatten(1, (hk, d)), proj[:, (h + hk) * d:].unflatten(1, (hk, d))
        s["k_cache"], s["v_cache"] = (torch.empty(n, cap, hk, d, dtype=BF16, device="cuda") for _ in range(2))
        s["k_cache"].normal_(generator=gen)
        s["v_cache"].normal_(generator=gen)
        return s
    if op == "append":
        hk, d = case["kv_heads"], case["dim"]
        proj = normal(n * t, 2 * hk * d)
        s["k_tree"], s["v_tree"] = (x.unflatten(1, (hk, d)) for x in proj.split([hk * d, hk * d], 1))
        cap = 48  # the rows' cost does not go by the cache's size
        s["len"] = torch.randint(0, cap - 8, (n,), generator=gen, device="cuda", dtype=torch.int32)
        s["len_out"] = torch.zeros_like(s["len"])
        s["k_cache"], s["v_cache"] = normal(n, cap, hk, d), normal(n, cap, hk, d)
        return s
    hk, hv = case["key_heads"], case["value_heads"]
    ch = (2 * hk + hv) * 128
    widths = [hk * 128, hk * 128, hv * 128, hv * 128, hv, hv]
    proj = normal(n * t, -(-sum(widths) // 8) * 8)[:, :sum(widths)]  # rows of whole 16 bytes
    s["q"], s["k"], s["v"], s["z"], s["a"], s["b"] = proj.split(widths, 1)
    s["conv_w"] = normal(ch, 4, std=0.5)
    s["A_log"] = torch.rand(hv, generator=gen, device="cuda") * math.log(16.0)
    s["norm_w"] = (1 + normal(128, std=0.1, dtype=torch.float32)).to(BF16)
    # the states lie in slots of a pool, in no order
    s["slots"] = n + 2
    s["slot"] = torch.randperm(s["slots"], generator=gen, device="cuda")[:n].to(torch.int32)
    s["state"] = normal(s["slots"], hv, 128, 128, std=0.1, dtype=torch.float32)
    s["conv"] = normal(s["slots"], 3, ch)
    if op == "commit":
        s["state_out"], s["conv_out"] = torch.zeros_like(s["state"]), torch.zeros_like(s["conv"])
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return {"rope": _rope, "attention": _attention, "delta": _delta, "commit": _commit, "append": _append}[s["case"]["op"]](s)


def _kept(s, name, make):
    """What a user's program makes once and keeps: the rotary table, the descriptor of fixed input buffers."""
    if name not in s:
        s[name] = make()
    return s[name]


def _inputs(s):
    from gated_delta_rule_81_b200 import gdn
    return _kept(s, "inputs", lambda: gdn.make_inputs(s["q"], s["k"], s["v"], s["a"], s["b"], s["z"], s["conv_w"], s["A_log"],
                                                      s["norm_w"]))


def _frequencies(case, dtype):
    """Turns a position makes, in radians, for each of the rotary_dim / 2 pairs, and the factor on cosine and sine."""
    r, base, factor = case["rotary"], case["base"], case["factor"]
    i = torch.arange(r // 2, dtype=dtype, device="cuda")
    if case["scaling"] == "ntk":
        base = base * factor ** (r / (r - 2))
    theta = torch.exp(i * (-2.0 / r * math.log(base)))
    if case["scaling"] == "linear":
        return theta / factor, 1.0
    if case["scaling"] != "yarn":
        return theta, 1.0
    # pairs that turn more than 32 times within the original length keep their frequency, fewer than once: divided
    def pair(turns):
        return r * math.log(_original(case) / (turns * 2 * math.pi)) / (2 * math.log(base))
    low, high = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), r // 2 - 1)
    ramp = ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
    return theta * (1 - ramp) + theta / factor * ramp, 0.1 * math.log(factor) + 1.0


def _original(case):
    """The length that scaled frequencies were made for."""
    return 32768


def _rope(s):
    c = s["case"]
    if own:
        from gated_delta_rule_81_b200 import gdn
        rope = _kept(s, "rope", lambda: gdn.make_rope(c["dim"], c["rotary"], base=c["base"], interleaved=c["interleaved"],
                                                      scaling=c["scaling"], factor=c["factor"], original_len=_original(c), eps=EPS))
        q, k, v = gdn.qk_norm_rope(rope, s["q"], s["k"], s["v"], q_norm_w=s["q_w"], k_norm_w=s["k_w"], positions=s["positions"],
                                   rows=s["rows"], k_out=s["k_out"], v_out=s["v_out"])
        return {"q": q, "k": k, "v": v}
    freq, mul = _frequencies(c, torch.float64)
    angle = s["positions"].double()[:, None] * freq  # far positions: 64 bits up to the reduced angle
    angle = (angle - torch.round(angle / (2 * math.pi)) * (2 * math.pi)).float()
    cos, sin = (angle.cos() * mul)[:, None], (angle.sin() * mul)[:, None]

    def turned(x, w):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        r = c["rotary"]
        x1, x2 = (x[..., 0:r:2], x[..., 1:r:2]) if c["interleaved"] else (x[..., :r // 2], x[..., r // 2:r])
        y1, y2 = x1 * cos - x2 * sin, x2 * cos + x1 * sin
        y = torch.stack([y1, y2], -1).flatten(-2) if c["interleaved"] else torch.cat([y1, y2], -1)
        return torch.cat([y, x[..., r:]], -1).to(BF16)

    s["k_out"][s["rows"]] = turned(s["k"], s["k_w"])
    s["v_out"][s["rows"]] = s["v"]
    return {"q": turned(s["q"], s["q_w"]), "k": s["k_out"], "v": s["v_out"]}


def _ancestors(parent):
    """live [N][T] and the closure [N][T][T] in 32 bits: 1 where column j is an ancestor of row t or t itself."""
    n, t = parent.shape
    p = parent.long()
    step = torch.arange(t, device=p.device)
    one = ((p[:, :, None] == step) & (step < step[:, None])).float()
    eye = torch.eye(t, device=p.device).expand(n, t, t)
    above = torch.linalg.solve_triangular(eye - one, eye, upper=False, unitriangular=True)  # I + P + P^2 + ...
    live = p >= -1
    return live, above * live[:, :, None] * live[:, None, :]


def _attention(s):
    c = s["case"]
    if own:
        from gated_delta_rule_81_b200 import gdn
        return gdn.attention_tree(s["q"], s["k_tree"], s["v_tree"], s["k_cache"], s["v_cache"], s["len"], s["parent"], g=s["g"])
    n, t, h, hk, d = c["seqs"], c["nodes"], c["heads"], c["kv_heads"], c["dim"]
    rows = int(s["k_cache"].shape[1])
    live, above = _ancestors(s["parent"])
    # [N][H_kv][T * group][D]: the queries that share a key head
    q = s["q"].float().view(n, t, hk, h // hk, d).permute(0, 2, 1, 3, 4).reshape(n, hk, -1, d) * d ** -0.5
    k, v = s["k_cache"].permute(0, 2, 1, 3).float(), s["v_cache"].permute(0, 2, 1, 3).float()
    kt, vt = (s[x].float().view(n, t, hk, d).permute(0, 2, 1, 3) for x in ("k_tree", "v_tree"))
    old = (q @ k.transpose(-1, -2)).masked_fill_(torch.arange(rows, device="cuda") >= s["len"][:, None, None, None], -math.inf)
    seen = above.repeat_interleave(h // hk, 1)[:, None] > 0
    new = (q @ kt.transpose(-1, -2)).masked_fill_(~seen, -math.inf)
    top = torch.maximum(old.amax(-1, keepdim=True), new.amax(-1, keepdim=True)).nan_to_num(neginf=0.0)
    old, new = old.sub_(top).exp_(), new.sub_(top).exp_()
    total = old.sum(-1, keepdim=True) + new.sum(-1, keepdim=True)
    o = (old @ v + new @ vt) / total.clamp(min=1e-30)
    o = o.view(n, hk, t, h // hk, d).permute(0, 2, 1, 3, 4).reshape(n, t, h, d) * live[:, :, None, None]
    if s["g"] is not None:
        o = o * torch.sigmoid(s["g"].float().view(n, t, h, d))
    return o.to(BF16).view(n * t, h * d)


def _features(s):
    """q, k [N][T][H_k][128] with norm 1, v [N][T][H_v][128], log decay and beta [N][T][H_v], and the raw rows
    behind three of history: the causal conv of each node runs along its own path."""
    c = s["case"]
    n, t, hk, hv = c["seqs"], c["nodes"], c["key_heads"], c["value_heads"]
    slot = s["slot"].long()
    raw = torch.cat([s["conv"][slot], torch.cat([s["q"], s["k"], s["v"]], 1).view(n, t, -1)], 1)
    # the row before each of the 3 + T rows: history in order, then parents
    p = s["parent"].long()
    before = torch.cat([torch.tensor([[0, 0, 1]], device="cuda").expand(n, 3), torch.where(p < 0, 2, p + 3)], 1)
    r3 = torch.arange(3, t + 3, device="cuda").expand(n, t)
    r2 = before.gather(1, r3)
    r1 = before.gather(1, r2)
    r0 = before.gather(1, r1)
    at = torch.arange(n, device="cuda")[:, None]
    w = s["conv_w"].float()
    y = raw[at, r0].float() * w[:, 0] + raw[at, r1].float() * w[:, 1] + raw[at, r2].float() * w[:, 2] + raw[at, r3].float() * w[:, 3]
    y = (y * torch.sigmoid(y)).unflatten(-1, (-1, 128))
    q, k, v = y.split([hk, hk, hv], 2)
    q, k = (x * torch.rsqrt((x * x).sum(-1, keepdim=True) + EPS) for x in (q, k))
    g = -s["A_log"].exp() * torch.nn.functional.softplus(s["a"].float())
    return q, k, v, g.view(n, t, hv), torch.sigmoid(s["b"].float()).view(n, t, hv), raw


def _writes(s, k, v, g, beta, state, live, above):
    """For each value head: the decay e^{G_t - G_j} [N][H][T][T], e^{G_t}, and u [N][H][T][128], where
    u_t = beta_t (v_t - e^{G_t} S k_t - sum over ancestors j of e^{G_t - G_j} (k_j . k_t) u_j)."""
    t, group = s["case"]["nodes"], s["case"]["value_heads"] // s["case"]["key_heads"]
    total = above.double() @ g.double()  # 64 bits: differences of long sums
    total = total.permute(0, 2, 1)
    decay = torch.exp((total[..., :, None] - total[..., None, :]).masked_fill(above[:, None] == 0, -math.inf)).float()
    start = total.exp().float()
    kh = k.permute(0, 2, 1, 3).repeat_interleave(group, 1)
    bt = (beta * live[:, :, None]).permute(0, 2, 1)[..., None]
    right = bt * (v.permute(0, 2, 1, 3) - start[..., None] * (kh @ state.transpose(-1, -2)))
    system = bt * decay * (kh @ kh.transpose(-1, -2)) * (1 - torch.eye(t, device="cuda")) + torch.eye(t, device="cuda")
    return decay, start, kh, torch.linalg.solve_triangular(system, right, upper=False, unitriangular=True)


def _delta(s):
    c = s["case"]
    n, t, hv = c["seqs"], c["nodes"], c["value_heads"]
    if own:
        from gated_delta_rule_81_b200 import gdn
        return gdn.decode_tree(_inputs(s), n, t, s["parent"], s["state"], s["conv"], state_slot=s["slot"])
    live, above = _ancestors(s["parent"])
    q, k, v, g, beta, _ = _features(s)
    state = s["state"][s["slot"].long()]
    decay, start, kh, u = _writes(s, k, v, g, beta, state, live, above)
    qh = q.permute(0, 2, 1, 3).repeat_interleave(hv // c["key_heads"], 1)
    o = start[..., None] * (qh @ state.transpose(-1, -2)) + (decay * (qh @ kh.transpose(-1, -2))) @ u
    o = o.permute(0, 2, 1, 3)
    z = s["z"].float().view(n, t, hv, 128)
    y = o * torch.rsqrt((o * o).mean(-1, keepdim=True) + EPS) * s["norm_w"].float() * (z * torch.sigmoid(z))
    return (y * live[:, :, None, None]).to(BF16).view(n * t, hv, 128)


def _path(s):
    """[N][T] in 32 bits: 1 on the accepted path."""
    _, above = _ancestors(s["parent"])
    last = s["accepted"].long()
    row = above.gather(1, last.clamp(min=0)[:, None, None].expand(-1, 1, above.shape[2]))[:, 0]
    return row * (last >= 0)[:, None]


def _commit(s):
    c = s["case"]
    n, t = c["seqs"], c["nodes"]
    if own:
        from gated_delta_rule_81_b200 import gdn
        gdn.decode_tree_commit(_inputs(s), n, t, s["parent"], s["accepted"], s["state"], s["conv"], state_slot=s["slot"],
                               state_out=s["state_out"], conv_out=s["conv_out"])
        return {"state": s["state_out"], "conv": s["conv_out"]}
    live, above = _ancestors(s["parent"])
    slot, last = s["slot"].long(), s["accepted"].long()
    q, k, v, g, beta, raw = _features(s)
    state = s["state"][slot]
    decay, start, kh, u = _writes(s, k, v, g, beta, state, live, above)
    at, some = last.clamp(min=0), (last >= 0)
    to_end = decay.gather(2, at[:, None, None, None].expand(-1, decay.shape[1], 1, t))[:, :, 0]  # e^{G_last - G_j}
    whole = start.gather(2, at[:, None, None].expand(-1, start.shape[1], 1))
    new = whole[..., None] * state + (u * to_end[..., None]).transpose(-1, -2) @ kh
    s["state_out"][slot] = torch.where(some[:, None, None, None], new, state)
    # the last three raw rows of history and path
    p = s["parent"].long()
    before = torch.cat([torch.tensor([[0, 0, 1]], device="cuda").expand(n, 3), torch.where(p < 0, 2, p + 3)], 1)
    r2 = torch.where(some, last + 3, 2)[:, None]
    r1 = before.gather(1, r2)
    r0 = before.gather(1, r1)
    s["conv_out"][slot] = raw[torch.arange(n, device="cuda")[:, None], torch.cat([r0, r1, r2], 1)]
    return {"state": s["state_out"], "conv": s["conv_out"]}


def _append(s):
    c = s["case"]
    n, t, hk, d = c["seqs"], c["nodes"], c["kv_heads"], c["dim"]
    if own:
        from gated_delta_rule_81_b200 import gdn
        gdn.attn_tree_commit(s["k_tree"], s["v_tree"], t, s["parent"], s["accepted"], s["k_cache"], s["v_cache"], s["len"],
                             cache_len_out=s["len_out"])
        return {"k": s["k_cache"], "v": s["v_cache"], "len": s["len_out"]}
    on = _path(s) > 0
    count = on.sum(1)
    to = s["len"].long()[:, None] + on.long().cumsum(1) - 1
    seq, node = on.nonzero(as_tuple=True)
    s["k_cache"][seq, to[seq, node]] = s["k_tree"].view(n, t, hk, d)[seq, node]
    s["v_cache"][seq, to[seq, node]] = s["v_tree"].view(n, t, hk, d)[seq, node]
    s["len_out"].copy_(s["len"] + count)
    return {"k": s["k_cache"], "v": s["v_cache"], "len": s["len_out"]}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "rope":
        n, d = case["tokens"], case["dim"]
        values = n * (case["heads"] + 2 * case["kv_heads"]) * d
        return {"bytes": 4 * values + 12 * n, "flops": 4 * n * (case["heads"] + case["kv_heads"]) * d}
    n, t = case["seqs"], case["nodes"]
    nodes = sum(_live(case))
    taken = sum(_accepted_nodes(case))
    if op == "attention":
        h, hk, d = case["heads"], case["kv_heads"], case["dim"]
        lens = _lengths(case)
        pairs = sum(a * b for a, b in zip(lens, _live(case)))
        per_node = (2 + (1 if case["gate"] else 0)) * h * d * 2 + 2 * hk * d * 2 + 4
        return {"bytes": sum(lens) * 2 * hk * d * 2 + nodes * per_node, "flops": 4 * d * h * pairs}
    if op == "append":
        return {"bytes": 4 * 2 * case["kv_heads"] * case["dim"] * taken + 4 * n * t + 12 * n, "flops": 0}
    hk, hv = case["key_heads"], case["value_heads"]
    state, ch = hv * 128 * 128 * 4, (2 * hk + hv) * 128
    if op == "delta":  # S k and S q of every node, its products with the nodes' keys and their sum
        return {"bytes": n * (state + 3 * ch * 2) + nodes * (ch + 2 * hv * 128 + 2 * hv) * 2 + ch * 8,
                "flops": nodes * (hv * 4 * 128 * 128 + hk * 2 * t * 128 + hv * 2 * t * 128)}
    return {"bytes": n * 2 * (state + 3 * ch * 2) + taken * (ch + 2 * hv) * 2 + ch * 8, "flops": taken * hv * 4 * 128 * 128}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    def rope(s):
        c = s["case"]
        n, d, r = c["tokens"], c["dim"], c["rotary"]
        base, factor, mul = c["base"], c["factor"], 1.0
        theta = []
        for i in range(r // 2):
            if c["scaling"] == "ntk":
                theta.append((base * factor ** (r / (r - 2))) ** (-2.0 * i / r))
            elif c["scaling"] == "linear":
                theta.append(base ** (-2.0 * i / r) / factor)
            else:
                theta.append(base ** (-2.0 * i / r))
        if c["scaling"] == "yarn":
            lo = r * math.log(32768 / (32.0 * 2 * math.pi)) / (2 * math.log(base))
            hi = r * math.log(32768 / (1.0 * 2 * math.pi)) / (2 * math.log(base))
            lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), r // 2 - 1)
            for i in range(r // 2):
                keep = 1.0 - min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
                theta[i] = theta[i] * keep + theta[i] / factor * (1.0 - keep)
            mul = 1.0 + 0.1 * math.log(factor)
        turn = torch.polar(torch.tensor(mul, dtype=torch.float64, device="cuda"),
                           s["positions"].double()[:, None, None] * torch.tensor(theta, dtype=torch.float64, device="cuda"))

        def head(x, w):
            x = x.double()
            x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / d + EPS) * w.double()
            a, b = (x[..., :r].unflatten(-1, (r // 2, 2)).unbind(-1) if c["interleaved"]
                    else x[..., :r].unflatten(-1, (2, r // 2)).unbind(-2))
            z = torch.complex(a.contiguous(), b.contiguous()) * turn
            y = torch.stack([z.real, z.imag], -1 if c["interleaved"] else -2).flatten(-2)
            return torch.cat([y, x[..., r:]], -1)

        k, v = s["k_out"].double(), s["v_out"].double()
        k.index_copy_(0, s["rows"], head(s["k"], s["k_w"]))
        v.index_copy_(0, s["rows"], s["v"].double())
        return {"q": head(s["q"], s["q_w"]), "k": k, "v": v}

    def walk(parent):
        """Each node's path from the first node to itself, for one sequence (a list of parents)."""
        paths = []
        for t, p in enumerate(parent):
            alive = p == -1 or (0 <= p < t and paths[p])
            paths.append(((paths[p] if p >= 0 else []) + [t]) if alive else [])
        return paths

    def attention(s):
        c = s["case"]
        n, t, h, hk, d = c["seqs"], c["nodes"], c["heads"], c["kv_heads"], c["dim"]
        group = h // hk
        out = torch.zeros(n, t, h, d, dtype=torch.float64, device="cuda")
        trees, lens = s["parent"].tolist(), s["len"].tolist()
        for i in range(n):
            bias = torch.full((t, t), -math.inf, dtype=torch.float64)
            paths = walk(trees[i])
            for node, path in enumerate(paths):
                bias[node, path] = 0.0
            there = [node for node, path in enumerate(paths) if path]
            bias = bias[there].cuda()
            for j in range(hk):
                keys = torch.cat([s["k_cache"][i, :lens[i], j], s["k_tree"][i * t:(i + 1) * t, j]]).double()
                values = torch.cat([s["v_cache"][i, :lens[i], j], s["v_tree"][i * t:(i + 1) * t, j]]).double()
                for e in range(group):
                    score = s["q"].view(n, t, h, d)[i, there, j * group + e].double() @ keys.T / math.sqrt(d)
                    score[:, lens[i]:] += bias
                    out[i, there, j * group + e] = torch.softmax(score, -1) @ values
        if s["g"] is not None:
            out = out / (1 + torch.exp(-s["g"].double().view(n, t, h, d)))
        return out.view(n * t, h * d)

    def recurrence(s):
        """The states of all nodes, one step of the rule after the other: [T + 1][N][H_v][128][128] with the
        committed state first, the outputs of each node, and the raw rows of each path's window of three."""
        c = s["case"]
        n, t, hk, hv = c["seqs"], c["nodes"], c["key_heads"], c["value_heads"]
        slot = s["slot"].long()
        raw = torch.cat([s["q"], s["k"], s["v"]], 1).double().view(n, t, -1)
        states = [s["state"][slot].double()]
        windows = [s["conv"][slot].double()]
        outs = []
        w = s["conv_w"].double()
        for step in range(t):
            p = s["parent"][:, step].long()
            which = [int(x) for x in p.clamp(min=-1).unique().tolist()]
            window, state = windows[0].clone(), states[0].clone()
            for x in which:
                mine = p == x
                window[mine], state[mine] = windows[x + 1][mine], states[x + 1][mine]
            full = torch.cat([window, raw[:, step:step + 1]], 1)
            y = (full * w.T).sum(1)
            y = (y / (1 + torch.exp(-y))).view(n, -1, 128)
            q, k, v = y[:, :hk], y[:, hk:2 * hk], y[:, 2 * hk:]
            q = (q / torch.sqrt((q ** 2).sum(-1, keepdim=True) + EPS)).repeat_interleave(hv // hk, 1)
            k = (k / torch.sqrt((k ** 2).sum(-1, keepdim=True) + EPS)).repeat_interleave(hv // hk, 1)
            a, b = s["a"].double().view(n, t, hv)[:, step], s["b"].double().view(n, t, hv)[:, step]
            alpha = torch.exp(-torch.exp(s["A_log"].double()) * torch.log1p(torch.exp(a)))
            beta = 1 / (1 + torch.exp(-b))
            state *= alpha[..., None, None]
            wrong = v - (state @ k[..., None])[..., 0]
            state += (beta[..., None] * wrong)[..., :, None] * k[..., None, :]
            o = (state @ q[..., None])[..., 0]
            z = s["z"].double().view(n, t, hv, 128)[:, step]
            y = o / torch.sqrt((o ** 2).mean(-1, keepdim=True) + EPS) * s["norm_w"].double() * z / (1 + torch.exp(-z))
            outs.append(y * (p >= -1)[:, None, None])
            states.append(state)
            windows.append(full[:, 1:])
        return states, windows, outs

    def delta(s):
        c = s["case"]
        _, _, outs = recurrence(s)
        return torch.stack(outs, 1).view(c["seqs"] * c["nodes"], c["value_heads"], 128)

    def commit(s):
        states, windows, _ = recurrence(s)
        state, conv = s["state_out"].double(), s["conv_out"].double()
        slot = s["slot"].long()
        for i, last in enumerate(s["accepted"].tolist()):
            state[slot[i]], conv[slot[i]] = states[last + 1][i], windows[last + 1][i]
        return {"state": state, "conv": conv}

    def append(s):
        c = s["case"]
        n, t, hk, d = c["seqs"], c["nodes"], c["kv_heads"], c["dim"]
        k, v, new = s["k_cache"].double(), s["v_cache"].double(), []
        for i, (tree, last, rows) in enumerate(zip(s["parent"].tolist(), s["accepted"].tolist(), s["len"].tolist())):
            path = walk(tree)[last] if last >= 0 else []
            for j, node in enumerate(path):
                k[i, rows + j], v[i, rows + j] = s["k_tree"][i * t + node].double(), s["v_tree"][i * t + node].double()
            new.append(rows + len(path))
        return {"k": k, "v": v, "len": None}

    return {"rope": rope, "attention": attention, "delta": delta, "commit": commit, "append": append}[case["op"]](prepare(case, seed))
