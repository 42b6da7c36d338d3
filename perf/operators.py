"""Cases of the serving operators: the layer core's step over cached states,
the recurrent gated delta rule alone, and the upkeep of the state cache.

A cache is one buffer of slots.  A slot holds, layer after layer, the fp32
state [hv][d][d] and the last three conv input rows [3][channels] (storage
type) of one sequence, each layer padded to 256 bytes.

kind "step":  conv -> gate -> gated delta rule -> gated norm for the next
              tokens of every sequence; states are read from slot_in, written
              to slot_out and, where slot_tok says so, after single tokens.
kind "rule":  the gated delta rule alone, on given q, k, v, g and beta.
kind "fork":  new slots are taken and filled with copies of others (or zeros),
              then given back, so that every pass does the same work.
kind "churn": some sequences end, the cache is compacted (the slot table of
              the running ones follows) and new sequences are admitted.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one user, the next token: latency
        dict(name="step_one", kind="step", hk=16, hv=48, d=128, dtype="bf16", seqs=1, empty=0,
             fresh=0, tokens=1, most=1, snap=False, inplace=True),
        # an ordinary batch of users, one token each
        dict(name="step_batch", kind="step", hk=16, hv=48, d=128, dtype="bf16", seqs=64, empty=0,
             fresh=0, tokens=64, most=1, snap=False, inplace=True),
        # a full batch: the states are far larger than any on-chip memory
        dict(name="step_full", kind="step", hk=16, hv=48, d=128, dtype="bf16", seqs=384, empty=0,
             fresh=0, tokens=384, most=1, snap=False, inplace=True),
        # draft tokens checked at once: one to eight a sequence, the state kept after each
        dict(name="step_drafts", kind="step", hk=16, hv=32, d=128, dtype="fp16", seqs=45, empty=0,
             fresh=0, tokens=203, most=8, snap=True, inplace=False),
        # one GPU's heads of four, a padded batch, some sequences new, each into another slot
        dict(name="step_padded", kind="step", hk=4, hv=8, d=128, dtype="bf16", seqs=37, empty=5,
             fresh=3, tokens=52, most=3, snap=False, inplace=False),
        # the smallest heads in fp32
        dict(name="rule_tiny", kind="rule", hk=1, hv=2, d=32, dtype="fp32", seqs=3, empty=0,
             fresh=1, tokens=11, most=7, snap=False, inplace=True),
        # one token each for many sequences
        dict(name="rule_batch", kind="rule", hk=16, hv=48, d=128, dtype="bf16", seqs=200, empty=0,
             fresh=0, tokens=200, most=1, snap=False, inplace=True),
        # a few sequences catch up on longer pieces, in fp32
        dict(name="rule_spans", kind="rule", hk=16, hv=32, d=128, dtype="fp32", seqs=7, empty=0,
             fresh=2, tokens=333, most=97, snap=False, inplace=True),
        # one conversation forks in two, on a small share of the heads
        dict(name="fork_small", kind="fork", hk=4, hv=8, d=128, dtype="bf16", layers=1, slots=16,
             live=5, copies=2, fresh=1),
        # a beam of copies and some new sequences, three layers' states to a slot
        dict(name="fork_large", kind="fork", hk=16, hv=48, d=128, dtype="bf16", layers=3, slots=120,
             live=61, copies=49, fresh=5),
        # two of eleven sequences are replaced
        dict(name="churn_small", kind="churn", hk=16, hv=32, d=128, dtype="bf16", layers=1,
             slots=16, live=11, ending=2),
        # a third of the sequences is replaced, two layers' states to a slot
        dict(name="churn_large", kind="churn", hk=16, hv=48, d=128, dtype="bf16", layers=2,
             slots=200, live=187, ending=60),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))


def draw(rng):
    kind = rng.choice(["step", "step", "rule", "rule", "fork", "churn"])
    d = rng.choice([32, 128, 128, 128])
    hk = rng.choice([1, 2, 3, 4, 8, 16])
    hv = hk * rng.choice([1, 2, 2, 3, 4])
    while hv > 48:
        hv -= hk
    c = dict(kind=kind, hk=hk, hv=hv, d=d, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    state = hv * d * d
    if kind in ("step", "rule"):
        snap = rng.random() < 0.3
        most = rng.choice([1, 1, 2, 4, 8]) if snap or rng.random() < 0.7 else _log(rng, 8, 80)
        room = 256 * 48 * 128 * 128 // state            # states kept, in all
        seqs = _log(rng, 1, min(384, max(1, room // (most + 1 if snap else 2))))
        if most > 8:
            seqs = min(seqs, 7)
        tokens = seqs if most == 1 else rng.randint(seqs, seqs * most)
        c.update(seqs=seqs, empty=rng.choice([0, 0, seqs // 7]), fresh=rng.choice([0, 0, seqs // 5]),
                 tokens=tokens, most=most, snap=snap, inplace=rng.random() < 0.5)
        c["tokens"] = min(c["tokens"], (seqs - c["empty"]) * most)
        c["tokens"] = max(c["tokens"], seqs - c["empty"])
    else:
        layers = rng.choice([1, 2, 3])
        room = max(8, 120 * 3 * 48 * 128 * 128 // (state * layers))
        slots = _log(rng, 8, min(400, room))
        if kind == "fork":
            live = rng.randint(1, max(1, slots // 2))
            copies = rng.randint(1, max(1, min(slots - live, 49 * 3 * 48 * 128 * 128 // (state * layers))))
            c.update(layers=layers, slots=slots, live=live, copies=copies,
                     fresh=rng.randint(0, min(5, slots - live - copies)))
        else:
            live = rng.randint(max(2, slots // 2), slots)
            ending = rng.randint(1, max(1, min(live // 2, 40 * 3 * 48 * 128 * 128 // (state * layers))))
            c.update(layers=layers, slots=slots, live=live, ending=ending)
    return c


# ------------------------------------------------------------------ the cache's layout
def _channels(c):
    return 2 * c["hk"] * c["d"] + c["hv"] * c["d"]


def _esize(c):
    return 4 if c["dtype"] == "fp32" else 2


def _layer_bytes(c):
    raw = c["hv"] * c["d"] * c["d"] * 4 + 3 * _channels(c) * _esize(c)
    return (raw + 255) // 256 * 256


def _views(buf, c, layer):
    """The layer's states [slots, hv, d, d] and conv rows [slots, 3, C]."""
    n, hv, d = buf.shape[0], c["hv"], c["d"]
    o0 = layer * _layer_bytes(c)
    o1 = o0 + hv * d * d * 4
    o2 = o1 + 3 * _channels(c) * _esize(c)
    S = buf[:, o0:o1].view(torch.float32).view(n, hv, d, d)
    C = buf[:, o1:o2].view(DTYPES[c["dtype"]]).view(n, 3, _channels(c))
    return S, C


def _lengths(c, rng):
    """Lengths of the sequences: `empty` of them zero, the others one to
    `most`, `tokens` in all."""
    n = c["seqs"] - c["empty"]
    lens = [1] * n
    open_ = list(range(n)) if c["most"] > 1 else []
    for _ in range(c["tokens"] - n):
        i = rng.randrange(len(open_))
        lens[open_[i]] += 1
        if lens[open_[i]] == c["most"]:
            open_[i] = open_[-1]
            open_.pop()
    lens += [0] * c["empty"]
    rng.shuffle(lens)
    return lens


def _slots_of(c):
    """Slots of a step's cache: those read, those written, a few others."""
    n = c["seqs"]
    return n + (0 if c["inplace"] else n) + (c["tokens"] if c["snap"] else 0) + 3


def prepare(case, seed):
    c = case
    dev = "cuda"
    rng = random.Random(seed)
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    hk, hv, d, C = c["hk"], c["hv"], c["d"], _channels(c)

    def n(*shape, std=1.0, to=torch.float32):
        return (torch.randn(shape, generator=gen, device=dev) * std).to(to)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    layers = c.get("layers", 1)
    slots = c["slots"] if "slots" in c else _slots_of(c)
    buf = torch.zeros(slots, layers * _layer_bytes(c), dtype=torch.uint8, device=dev)
    for k in range(layers):
        S, cr = _views(buf, c, k)
        S.normal_(0.0, 0.1, generator=gen)
        cr.copy_(n(slots, 3, C, to=dt))
    s = dict(case=c, buf=buf)

    if c["kind"] in ("step", "rule"):
        lens = _lengths(c, rng)
        T, N = sum(lens), len(lens)
        order = list(range(slots))
        rng.shuffle(order)
        slot_in = order[:N]
        slot_out = list(slot_in) if c["inplace"] else order[N:2 * N]
        rest = order[N if c["inplace"] else 2 * N:]
        full = [i for i in range(N) if lens[i]]
        for i in range(N):
            if lens[i] == 0:
                slot_in[i] = slot_out[i] = -1     # padding of the batch
        for i in rng.sample(full, min(c["fresh"], len(full))):
            slot_in[i] = -1                       # a new sequence: the zero state
        cu = [0]
        for x in lens:
            cu.append(cu[-1] + x)
        s.update(cu=ints(cu), most=max(lens), slot_in=ints(slot_in), slot_out=ints(slot_out),
                 slot_tok=ints(rest[:T]) if c["snap"] else None)
        # the gate's parameters: decay rates 1..16 and time steps 0.001..0.1, as such layers start
        A_log = torch.log(1 + 15 * torch.rand(hv, generator=gen, device=dev))
        dts = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(hv, generator=gen, device=dev))
        dt_bias = torch.log(torch.expm1(dts))
        if c["kind"] == "step":
            s.update(x=n(T, C, to=dt), w_conv=n(C, 4, std=0.25), a=n(T, hv, to=dt), b=n(T, hv, to=dt),
                     A_log=A_log, dt_bias=dt_bias, z=n(T, hv, d, to=dt), w_norm=n(d, std=0.1))
        else:
            y = n(T, C)
            qk = y[:, :2 * hk * d].reshape(T, 2 * hk, d)
            y[:, :2 * hk * d] = (qk / qk.square().sum(-1, keepdim=True).sqrt()).reshape(T, -1)
            y = y.to(dt)
            g = -torch.exp(A_log) * torch.nn.functional.softplus(n(T, hv) + dt_bias)
            s.update(q=y[:, :hk * d], k=y[:, hk * d:2 * hk * d], v=y[:, 2 * hk * d:], g=g,
                     beta=torch.sigmoid(n(T, hv)))
    elif c["kind"] == "fork":
        live = rng.sample(range(slots), c["live"])
        refs = [0] * slots
        for i in live:
            refs[i] = rng.choice([1, 1, 2])
        src = [rng.choice(live) for _ in range(c["copies"])] + [-1] * c["fresh"]
        rng.shuffle(src)
        s.update(refs=ints(refs), src=ints(src))
    else:
        live, ending = c["live"], c["ending"]
        refs = [1] * live + [0] * (slots - live)
        table = list(range(live))
        rng.shuffle(table)
        s.update(refs=ints(refs), table=ints(table), src=ints([-1] * ending),
                 ending=ints(rng.sample(range(live - ending), ending)))
    if own:
        from gated_deltanet_layer_causal_amd.layer import CoreConfig, GDNCore, GDNStateCache
        s["core"] = GDNCore(CoreConfig(hk=hk, hv=hv, d=d, dtype=dt), device=dev)
        s["cache"] = GDNStateCache(s["core"].cfg, slots, n_layers=layers, device=dev, buffer=buf,
                                   refs=s.get("refs"))
    return s


# ------------------------------------------------------------------ plain forms
def _rule_token(S, q, k, v, g, beta):
    """One token of the rule for the states S [M, hv, d, d]."""
    S = S * torch.exp(g)[:, :, None, None]
    delta = beta[:, :, None] * (v - (S * k[:, :, None, :]).sum(-1))
    S = S + delta[..., None] * k[:, :, None, :]
    return S, (S * q[:, :, None, :]).sum(-1)


def _put(pool, slots, rows):
    keep = slots >= 0
    pool[slots[keep].long()] = rows[keep].to(pool.dtype)


def _take(pool, slots):
    got = pool[slots.clamp(min=0).long()].float()
    got[slots < 0] = 0
    return got


def _plain_recurrence(s, c, hist, tokens_of, S_pool, C_pool):
    """Walks all sequences token by token.  tokens_of(at, rows) gives q, k, v, g, beta
    of the tokens `at` and, for the step, updates the conv windows of `rows`."""
    hv, d = c["hv"], c["d"]
    G = hv // c["hk"]
    start, lens = s["cu"][:-1].long(), s["cu"].diff()
    S = _take(S_pool, s["slot_in"])
    o = torch.empty(int(c["tokens"]), hv, d, device=S.device)
    one = s["most"] == 1 and c["empty"] == 0
    for j in range(s["most"]):
        rows = slice(None) if one else (lens > j).nonzero()[:, 0]
        at = start[rows] + j
        q, k, v, g, beta = tokens_of(at, rows)
        new, ot = _rule_token(S[rows], q.repeat_interleave(G, 1), k.repeat_interleave(G, 1), v, g, beta)
        o[at] = ot
        if one:
            S = new
        else:
            S[rows] = new
        if s["slot_tok"] is not None:
            _put(S_pool, s["slot_tok"][at], new)
            if hist is not None:
                _put(C_pool, s["slot_tok"][at], hist[rows])
    _put(S_pool, s["slot_out"], S)
    if hist is not None:
        _put(C_pool, s["slot_out"], hist)
    return o


def _plain_step(s):
    c = s["case"]
    hk, hv, d = c["hk"], c["hv"], c["d"]
    S_pool, C_pool = _views(s["buf"], c, 0)
    hist = _take(C_pool, s["slot_in"])

    def tokens_of(at, rows):
        M = at.numel()
        win = torch.cat([hist[rows], s["x"][at].float()[:, None]], 1)
        hist[rows] = win[:, 1:]
        u = (win * s["w_conv"].t()).sum(1)
        y = u / (1 + torch.exp(-u))
        q, k, v = y.split([hk * d, hk * d, hv * d], 1)
        q, k, v = q.view(M, hk, d), k.view(M, hk, d), v.reshape(M, hv, d)
        q = q / (q.square().sum(-1, keepdim=True) + 1e-6).sqrt() * d ** -0.5
        k = k / (k.square().sum(-1, keepdim=True) + 1e-6).sqrt()
        xa = s["a"][at].float() + s["dt_bias"]
        g = -torch.exp(s["A_log"]) * (xa.clamp(min=0) + torch.log1p(torch.exp(-xa.abs())))
        return q, k, v, g, 1 / (1 + torch.exp(-s["b"][at].float()))

    o = _plain_recurrence(s, c, hist, tokens_of, S_pool, C_pool)
    z = s["z"].float()
    out = o / (o.square().mean(-1, keepdim=True) + 1e-6).sqrt() * (1 + s["w_norm"])
    out = (out * z / (1 + torch.exp(-z))).to(s["x"].dtype)
    return {"out": out, "S": S_pool, "conv": C_pool}


def _plain_rule(s):
    c = s["case"]
    hk, hv, d = c["hk"], c["hv"], c["d"]
    S_pool, _ = _views(s["buf"], c, 0)

    def tokens_of(at, rows):
        M = at.numel()
        return (s["q"][at].float().view(M, hk, d) * d ** -0.5, s["k"][at].float().view(M, hk, d),
                s["v"][at].float().view(M, hv, d), s["g"][at], s["beta"][at])

    o = _plain_recurrence(s, c, None, tokens_of, S_pool, None)
    return {"o": o.to(s["q"].dtype), "S": S_pool}


def _plain_fork(buf, refs, src):
    n = refs.numel()
    free = (refs == 0).nonzero()[:, 0]
    known = (src >= 0) & (src < n)
    valid = (src == -1) | (known & (refs[src.clamp(0, n - 1).long()] > 0))
    rank = valid.cumsum(0) - 1
    given = valid & (rank < free.numel())
    dst = torch.full_like(src, -1)
    dst[given] = free[rank[given]].to(torch.int32)
    copy, zero = given & (src >= 0), given & (src < 0)
    buf[dst[copy].long()] = buf[src[copy].long()]
    buf[dst[zero].long()] = 0
    refs[dst[given].long()] = 1
    return dst


def _plain_release(refs, slots):
    refs.index_add_(0, slots.long(), torch.full_like(slots, -1))
    refs.clamp_(min=0)


def _plain_compact(buf, refs, table):
    n = refs.numel()
    live = refs > 0
    L = live.sum()
    at = torch.arange(n, device=refs.device)
    holes = (~live & (at < L)).nonzero()[:, 0]
    movers = (live & (at >= L)).nonzero()[:, 0]
    buf[holes] = buf[movers]
    remap = torch.where(live, at, torch.full_like(at, -1)).to(torch.int32)
    remap[movers] = holes.to(torch.int32)
    refs[holes] = refs[movers]
    refs[movers] = 0
    table.copy_(remap[table.long()])
    return remap


def run(state):
    s = state
    c, kind = s["case"], s["case"]["kind"]
    if own:
        core, cache = s["core"], s["cache"]
        if kind == "step":
            out = core.step(s["x"], s["w_conv"], s["a"], s["b"], s["A_log"], s["dt_bias"], s["z"],
                            s["w_norm"], s["cu"], cache, s["slot_in"], s["slot_out"], s["slot_tok"])
            return {"out": out, "S": cache.S(0), "conv": cache.conv(0)}
        if kind == "rule":
            o = core.recurrent(s["q"], s["k"], s["v"], s["g"], s["beta"], s["cu"], cache,
                               s["slot_in"], s["slot_out"], s["slot_tok"])
            return {"o": o, "S": cache.S(0)}
        if kind == "fork":
            dst = cache.fork(s["src"])
            cache.release(dst)
            return {"slots": dst, "refs": s["refs"], "cache": s["buf"].view(torch.int32)}
        cache.release(s["ending"])
        remap = cache.compact(s["table"])
        dst = cache.fork(s["src"])
    else:
        if kind == "step":
            return _plain_step(s)
        if kind == "rule":
            return _plain_rule(s)
        if kind == "fork":
            dst = _plain_fork(s["buf"], s["refs"], s["src"])
            _plain_release(s["refs"], dst)
            return {"slots": dst, "refs": s["refs"], "cache": s["buf"].view(torch.int32)}
        _plain_release(s["refs"], s["ending"])
        remap = _plain_compact(s["buf"], s["refs"], s["table"])
        dst = _plain_fork(s["buf"], s["refs"], s["src"])
    # the admitted sequences take the places of those that ended
    s["table"].masked_scatter_(s["table"] < 0, dst)
    return {"remap": remap, "slots": dst, "table": s["table"], "refs": s["refs"],
            "cache": s["buf"].view(torch.int32)}


def work(case):
    c = case
    hk, hv, d, C, E = c["hk"], c["hv"], c["d"], _channels(c), _esize(c)
    S_bytes, conv_bytes = hv * d * d * 4, 3 * C * E
    if c["kind"] in ("step", "rule"):
        full, T = c["seqs"] - c["empty"], c["tokens"]
        states = 2 * full - min(c["fresh"], full) + (T if c["snap"] else 0)
        if c["kind"] == "step":
            tok = T * (C * E + 2 * hv * E + 2 * hv * d * E)
            return {"bytes": states * (S_bytes + conv_bytes) + tok + C * 16 + hv * 8 + d * 4,
                    "flops": T * (hv * 8 * d * d + C * 8 + hv * d * 8)}
        return {"bytes": states * S_bytes + T * (C * E + hv * d * E + hv * 8),
                "flops": T * hv * 8 * d * d}
    slot = c["layers"] * _layer_bytes(c)
    if c["kind"] == "fork":
        n = c["copies"] + c["fresh"]
        return {"bytes": (2 * c["copies"] + c["fresh"]) * slot + 8 * c["slots"] + 8 * n, "flops": 0}
    return {"bytes": 3 * c["ending"] * slot + 12 * c["slots"] + 8 * c["live"], "flops": 0}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    """Sequence by sequence and token by token, from
    S_t = e^g S_{t-1} (I - beta k k^T) + beta v k^T and o_t = S_t q_t."""
    c = case
    if c["kind"] in ("fork", "churn"):
        return None                       # whole numbers and copies: compared as they are
    if c["tokens"] > 4000:
        return None
    s = prepare(case, seed)
    f = torch.float64
    hk, hv, d = c["hk"], c["hv"], c["d"]
    Sp, Cp = _views(s["buf"], c, 0)
    S_new, C_new = Sp.to(f), Cp.to(f)
    cu, si, so = s["cu"].tolist(), s["slot_in"].tolist(), s["slot_out"].tolist()
    st = s["slot_tok"].tolist() if s["slot_tok"] is not None else None
    dev = Sp.device
    head = torch.arange(hv, device=dev) // (hv // hk)
    outs = torch.zeros(c["tokens"], hv, d, dtype=f, device=dev)
    step = c["kind"] == "step"
    for i in range(c["seqs"]):
        t0, t1 = cu[i], cu[i + 1]
        S = Sp[si[i]].to(f) if si[i] >= 0 else torch.zeros(hv, d, d, dtype=f, device=dev)
        if step:
            before = Cp[si[i]].to(f) if si[i] >= 0 else torch.zeros(3, _channels(c), dtype=f, device=dev)
            line = torch.cat([before, s["x"][t0:t1].to(f)], 0)
        for t in range(t0, t1):
            if step:
                w = s["w_conv"].to(f)
                u = sum(line[t - t0 + j] * w[:, j] for j in range(4))
                y = u * torch.sigmoid(u)
                q = y[:hk * d].reshape(hk, d)
                k = y[hk * d:2 * hk * d].reshape(hk, d)
                v = y[2 * hk * d:].reshape(hv, d)
                q = q * torch.rsqrt((q * q).sum(1, keepdim=True) + 1e-6)
                k = k * torch.rsqrt((k * k).sum(1, keepdim=True) + 1e-6)
                xa = s["a"][t].to(f) + s["dt_bias"].to(f)
                g = -torch.exp(s["A_log"].to(f)) * torch.logaddexp(xa, torch.zeros_like(xa))
                beta = torch.sigmoid(s["b"][t].to(f))
            else:
                q, k = s["q"][t].to(f).view(hk, d), s["k"][t].to(f).view(hk, d)
                v, g, beta = s["v"][t].to(f).view(hv, d), s["g"][t].to(f), s["beta"][t].to(f)
            q, k = q[head] / math.sqrt(d), k[head]
            Sk = (S * k[:, None, :]).sum(2)
            S = torch.exp(g)[:, None, None] * (S - (beta[:, None] * Sk)[:, :, None] * k[:, None, :]) \
                + (beta[:, None] * v)[:, :, None] * k[:, None, :]
            o = (S * q[:, None, :]).sum(2)
            if step:
                z = s["z"][t].to(f)
                o = o * torch.rsqrt((o * o).mean(1, keepdim=True) + 1e-6) * (1 + s["w_norm"].to(f))
                o = o * z * torch.sigmoid(z)
            outs[t] = o
            if st is not None and st[t] >= 0:
                S_new[st[t]] = S
                if step:
                    C_new[st[t]] = line[t - t0 + 1:t - t0 + 4]
        if so[i] >= 0:
            S_new[so[i]] = S
            if step:
                C_new[so[i]] = line[t1 - t0:t1 - t0 + 3]
    return {"out": outs, "S": S_new, "conv": C_new} if step else {"o": outs, "S": S_new}
