"""The operators that serve several continuations and encoders beside the hybrid layer, as measured.

fork    the memories of a layer's sequences copied to other sequences: the samples of one
        prompt, the beams that survive a step (in place), the sequences that are not finished.
        For sequence b of the result and every memory x: x'[b] = x[parents[b]].
cross   attention of T decoder tokens to an encoder's S states of another length, grouped heads:
        y[b,t,h] = sum_s p_s v[b,s,g],  p = softmax_s(scale q[b,t,h].k[b,s,g]) over s < kv_len[b],
        g = h // (Hq / Hkv); a sequence with kv_len 0 reads nothing and gets y = 0.
prefix  attention of a batch whose sequences share a prefix of P keys, each followed by keys of
        its own: query t of sequence b reads every prefix key and its own keys
        s <= own_len[b] - T + t, under one softmax.

`own` chooses between the plain forms in torch and the calls of this repository's package.
"""
import math
import random

import torch

own = False

MEMORIES = ("H", "s", "cache_k", "cache_v", "cache_phik", "cache_pos", "win_k", "win_v", "win_phik")
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ---------------------------------------------------------------------------------

def _fork(name, kind, B, n, Hq, Hkv, d, Dh, eta, lam, chunk, dtype):
    """kind "samples": B prompts to n sequences; "beams": n of B sequences live on, in place;
    "compact": n of B sequences kept."""
    return dict(name=name, op="fork", kind=kind, B=B, n=n, Hq=Hq, Hkv=Hkv, d=d, Dh=Dh, eta=eta, lam=lam,
                chunk=chunk, dtype=dtype)


def _cross(name, B, T, S, Hq, Hkv, d, dtype, lens):
    """lens "full": every sequence has S states; "ragged": S/2 to S; "empty": ragged, one with none."""
    return dict(name=name, op="cross", B=B, T=T, S=S, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, lens=lens)


def _prefix(name, B, T, P, L, Hq, Hkv, d, dtype, lens):
    """lens: as in _cross, of the sequences' own keys (L at most, the queries' own among them)."""
    return dict(name=name, op="prefix", B=B, T=T, P=P, L=L, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, lens=lens)


def listed():
    return [
        # a small f32 layer's four sequences, one finished: what a call costs at least
        _fork("fork-compact-small", "compact", 4, 3, 1, 1, 64, 32, 64, 64, 64, "f32"),
        # one prompt prefilled once, then 64 samples of it (the decode workload's layer)
        _fork("fork-samples-64", "samples", 1, 64, 32, 8, 128, 64, 64, 256, 64, "bf16"),
        # a step of a beam search: 20 of 64 beams live on in place
        _fork("fork-beams-64", "beams", 64, 20, 32, 8, 128, 64, 64, 256, 64, "bf16"),
        # one token against a short caption's states: what a call costs at least
        _cross("cross-token-small", 1, 1, 77, 32, 8, 128, "bf16", "full"),
        # one token of each of 64 sequences against audio-sized states, padded
        _cross("cross-token-64", 64, 1, 1500, 32, 8, 128, "bf16", "empty"),
        # a decoder's prompt against a document's states
        _cross("cross-prompt-4k", 4, 4096, 4096, 32, 8, 128, "bf16", "ragged"),
        # a small model in f32, odd lengths, three query heads to a kv head
        _cross("cross-prompt-f32", 2, 333, 1001, 12, 4, 64, "f32", "ragged"),
        # two samples of a short prompt: what a call costs at least
        _prefix("prefix-token-small", 2, 1, 200, 17, 32, 8, 128, "bf16", "full"),
        # a token of each of 64 samples that share a long document
        _prefix("prefix-token-64", 64, 1, 16384, 512, 32, 8, 128, "bf16", "ragged"),
        # five drafted tokens of each of 16 samples, odd lengths, the smaller head
        _prefix("prefix-draft-16", 16, 5, 8191, 257, 32, 8, 64, "bf16", "empty"),
        # 8 questions of 512 tokens about one document
        _prefix("prefix-prompt-8", 8, 512, 8192, 512, 32, 8, 128, "bf16", "full"),
        # a small f32 layer, a token of each of 7 samples
        _prefix("prefix-token-f32", 7, 1, 4095, 130, 6, 2, 64, "f32", "ragged"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    dtype = rng.choice(("bf16", "bf16", "f32"))
    d = rng.choice((64, 128))
    Hkv = rng.choice((1, 2, 4, 8))
    Hq = Hkv * rng.randint(1, 8)
    op = rng.choice(("fork", "cross", "prefix"))
    if op == "fork":
        eta, lam = _log(rng, 3, 300), _log(rng, 4, 512)
        per = Hkv * (eta + lam) * (2 * d + 128) * 4
        B = _log(rng, 2, max(2, min(64, 150_000_000 // per)))
        kind = rng.choice(("samples", "beams", "compact"))
        n = rng.randint(1, B)
        c = _fork("", kind, n if kind == "samples" else B, B if kind == "samples" else n, Hq, Hkv, d,
                  rng.choice((32, 64)), eta, lam, 16, dtype)
    else:
        lens = rng.choice(("full", "ragged", "empty"))
        B, T = _log(rng, 1, 64), rng.choice((1, 1, rng.randint(2, 9), _log(rng, 10, 2048)))
        # (f32: a hundredth of the largest listed case's products)
        most = (5e11 if dtype == "bf16" else 5e9) / (4.0 * Hq * d)
        B = max(1, min(B, int(most / T / 64)))
        T = max(1, min(T, int(most / B / 64), int(5e7 / (B * Hq * d))))
        keys = max(2, min(16384, int(most / B / T), int(5e7 / (B * Hkv * d))))
        if op == "cross":
            c = _cross("", B, T, _log(rng, 1, keys), Hq, Hkv, d, dtype, lens)
        else:
            P = _log(rng, 1, keys)
            L = T + _log(rng, 1, max(1, min(1024, keys - T)))
            c = _prefix("", B, T, P, L, Hq, Hkv, d, dtype, lens)
    del c["name"]
    return c


def _lens(case, n):
    """The lengths of a batch, at most n, before they are dealt to the sequences."""
    B = case["B"]
    if case["lens"] == "full":
        return [n] * B
    got = [n - (n // 2) * i // max(1, B - 1) for i in range(B)]
    if case["lens"] == "empty" and B > 1:
        got[-1] = 0
    return got


def _moves(case):
    """(sequences read, sequences written) of a fork."""
    B, n = case["B"], case["n"]
    if case["kind"] == "beams":
        return min(n, B - n), B - n
    return (min(B, n) if case["kind"] == "samples" else n), n


def _parents(case, seed):
    r, B, n = random.Random(seed), case["B"], case["n"]
    if case["kind"] == "samples":
        return [i * B // n for i in range(n)]
    live = sorted(r.sample(range(B), n))
    if case["kind"] == "compact":
        return live
    r.shuffle(live)
    dead = sorted(set(range(B)) - set(live))
    got = list(range(B))
    for j, b in enumerate(dead):
        got[b] = live[j % n]
    return got


# ---- inputs --------------------------------------------------------------------------------

def _memories(case, seed):
    """Memories as a prompt leaves them: feature rows are positive and sum to 2, positions distinct."""
    g = torch.Generator("cuda").manual_seed(seed)
    N, d, D, lam, eta = case["B"] * case["Hkv"], case["d"], 2 * case["Dh"], case["lam"], case["eta"]
    t = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def phi(rows):
        z = normal(N, rows, D // 2)
        return torch.cat([torch.softmax(z, -1), torch.softmax(-z, -1)], -1)

    return dict(H=normal(N, D, d), s=normal(N, D).square(), cache_k=normal(N, lam, d).to(t),
                cache_v=normal(N, lam, d).to(t), cache_phik=phi(lam),
                cache_pos=torch.argsort(normal(N, lam), 1).to(torch.int32),
                win_k=normal(N, eta, d).to(t), win_v=normal(N, eta, d).to(t), win_phik=phi(eta))


def _layer(case, B, mem=None):
    """A layer of this repository with room for B sequences; with `mem`, after a prompt that left these memories."""
    import sparse_kv_caching_b200 as lola
    c, t = case, TYPES[case["dtype"]]
    T = -(-(c["eta"] + c["lam"]) // c["chunk"]) * c["chunk"] if mem else c["chunk"]
    cfg = lola.make_config(B, c["Hq"], c["Hkv"], c["d"], c["Dh"], c["eta"], c["lam"], c["chunk"], c["dtype"], T)
    layer = lola.LolaLayer(cfg, torch.zeros(c["Hkv"], c["d"], c["Dh"], dtype=t, device="cuda"))
    if mem:
        q = torch.zeros(B, T, c["Hq"], c["d"], dtype=t, device="cuda")
        k = torch.zeros(B, T, c["Hkv"], c["d"], dtype=t, device="cuda")
        layer.prefill(q, k, k)
        if c["kind"] == "beams":        # a search forks between decode steps
            layer.decode(q[:, 0].contiguous(), k[:, 0].contiguous(), k[:, 0].contiguous())
        views = layer.export()
        for name in MEMORIES:
            views[name].copy_(mem[name])
    return layer


def prepare(case, seed):
    if case["op"] == "fork":
        parents = torch.tensor(_parents(case, seed), dtype=torch.int32, device="cuda")
        mem = _memories(case, seed)
        n, in_place = parents.numel(), case["kind"] == "beams"
        st = dict(case=case, parents=parents, in_place=in_place)
        if own:
            st["src"] = _layer(case, case["B"], mem)
            st["dst"] = st["src"] if in_place else _layer(case, n)
            views = st["dst"].export()
            st["out"] = {name: views[name] for name in MEMORIES}
        else:
            st["index"] = parents.long()
            st["src"] = mem
            st["out"] = mem if in_place else {
                name: torch.empty((n * case["Hkv"],) + x.shape[1:], dtype=x.dtype, device="cuda")
                for name, x in mem.items()}
        return st
    g = torch.Generator("cuda").manual_seed(seed)
    B, T, Hq, Hkv, d, t = (case[x] for x in ("B", "T", "Hq", "Hkv", "d", "dtype"))

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(TYPES[t])

    lens = _lens(case, case["S"] if case["op"] == "cross" else case["L"])
    random.Random(seed).shuffle(lens)
    st = dict(case=case, q=normal(B, T, Hq, d))
    n = torch.tensor(lens, dtype=torch.int32, device="cuda") if case["lens"] != "full" else None
    if case["op"] == "cross":
        st.update(k=normal(B, case["S"], Hkv, d), v=normal(B, case["S"], Hkv, d), kv_len=n)
    else:
        st.update(k_prefix=normal(case["P"], Hkv, d), v_prefix=normal(case["P"], Hkv, d),
                  k_own=normal(B, case["L"], Hkv, d), v_own=normal(B, case["L"], Hkv, d), own_len=n)
    return st


# ---- one pass ------------------------------------------------------------------------------

def _plain_fork(st):
    Hkv = st["case"]["Hkv"]
    for name in MEMORIES:
        x, y = st["src"][name], st["out"][name]
        moved = x.view(-1, Hkv, *x.shape[1:])[st["index"]]
        y.view(-1, Hkv, *y.shape[1:]).copy_(moved)
    return st["out"]


def _rows(x, Hkv):
    """[B, T, Hq, d] as [B, Hkv, T * Gq, d] in f32: the rows that read one kv head."""
    B, T, Hq, d = x.shape
    return x.float().view(B, T, Hkv, Hq // Hkv, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * (Hq // Hkv), d)


def _back(y, q):
    B, T, Hq, d = q.shape
    Hkv = y.shape[1]
    return y.view(B, Hkv, T, Hq // Hkv, d).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, d).to(q.dtype)


def _plain_cross(st):
    q, k, v = st["q"], st["k"], st["v"]
    S, Hkv, d = k.shape[1:]
    w = _rows(q, Hkv) @ k.float().permute(0, 2, 3, 1) / math.sqrt(d)
    if st["kv_len"] is not None:
        seen = torch.arange(S, device=q.device) < st["kv_len"][:, None]
        w = w.masked_fill(~seen[:, None, None, :], -math.inf)
    top = w.amax(-1, keepdim=True)
    w = torch.exp(w - torch.where(top == -math.inf, 0.0, top))
    total = w.sum(-1, keepdim=True)
    y = w @ v.float().permute(0, 2, 1, 3)
    return _back(torch.where(total > 0, y / total, 0.0), q)


def _plain_prefix(st):
    q, kp, vp, ko, vo = (st[x] for x in ("q", "k_prefix", "v_prefix", "k_own", "v_own"))
    B, T, Hq, d = q.shape
    L, Hkv = ko.shape[1:3]
    rows = _rows(q, Hkv) / math.sqrt(d)
    shared = rows.permute(1, 0, 2, 3).reshape(Hkv, -1, d) @ kp.float().permute(1, 2, 0)    # [Hkv, B T Gq, P]
    mine = rows @ ko.float().permute(0, 2, 3, 1)                                           # [B, Hkv, T Gq, L]
    n = st["own_len"][:, None] if st["own_len"] is not None else torch.full((B, 1), L, device=q.device)
    sees = n - T + 1 + torch.arange(T, device=q.device)                                    # [B, T] own keys read
    seen = torch.arange(L, device=q.device) < sees.repeat_interleave(Hq // Hkv, 1)[..., None]
    mine = mine.masked_fill(~seen[:, None], -math.inf)
    shared = shared.view(Hkv, B, -1, shared.shape[-1]).transpose(0, 1)
    top = torch.maximum(shared.amax(-1, keepdim=True), mine.amax(-1, keepdim=True))
    shared, mine = torch.exp(shared - top), torch.exp(mine - top)
    total = shared.sum(-1, keepdim=True) + mine.sum(-1, keepdim=True)
    y = shared.transpose(0, 1).reshape(Hkv, -1, shared.shape[-1]) @ vp.float().permute(1, 0, 2)
    y = y.view(Hkv, B, -1, d).transpose(0, 1) + mine @ vo.float().permute(0, 2, 1, 3)
    return _back(y / total, q)


def run(st):
    op = st["case"]["op"]
    if not own:
        return {"fork": _plain_fork, "cross": _plain_cross, "prefix": _plain_prefix}[op](st)
    import sparse_kv_caching_b200 as lola
    if op == "fork":
        st["dst"].fork(st["parents"], src=st["src"])
        return st["out"]
    if op == "cross":
        return lola.cross_attention(st["q"], st["k"], st["v"], kv_len=st["kv_len"])
    return lola.prefix_attention(st["q"], st["k_prefix"], st["v_prefix"], st["k_own"], st["v_own"],
                                 own_len=st["own_len"])


# ---- what a pass cannot do without -----------------------------------------------------------

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    Hkv, d = case["Hkv"], case["d"]
    if case["op"] == "fork":
        D = 2 * case["Dh"]
        per = D * d * 4 + D * 4 + (case["lam"] + case["eta"]) * (2 * d * e + D * 4) + case["lam"] * 4
        return {"bytes": sum(_moves(case)) * Hkv * per, "flops": 0}
    B, T, Hq = case["B"], case["T"], case["Hq"]
    move = 2 * B * T * Hq * d * e
    if case["op"] == "cross":
        lens = _lens(case, case["S"])
        return {"bytes": move + 2 * sum(lens) * Hkv * d * e, "flops": 4 * T * sum(lens) * Hq * d}
    lens = _lens(case, case["L"])
    pairs = sum(case["P"] + max(0, n - T + 1 + t) for n in lens for t in range(T))
    return {"bytes": move + 2 * (case["P"] + sum(lens)) * Hkv * d * e, "flops": 4 * pairs * Hq * d}


# ---- the definition in 64 bits ---------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "fork":
        mem = _memories(case, seed)
        Hkv, rows = case["Hkv"], []
        for p in _parents(case, seed):
            rows += range(p * Hkv, (p + 1) * Hkv)
        return {name: torch.stack([x[i] for i in rows]).to(torch.float64 if x.is_floating_point() else x.dtype)
                for name, x in mem.items()}
    st = prepare(case, seed)
    q = st["q"].double()
    B, T, Hq, d = q.shape
    Gq = Hq // case["Hkv"]
    y = torch.zeros_like(q)
    own_len = st.get("own_len", st.get("kv_len"))
    lens = own_len.tolist() if own_len is not None else [case["S"] if case["op"] == "cross" else case["L"]] * B
    for b in range(B):
        for g in range(case["Hkv"]):
            if case["op"] == "cross":
                k, v = (st[x][b, :lens[b], g].double() for x in ("k", "v"))
                if lens[b] == 0:
                    continue
            else:
                k = torch.cat([st["k_prefix"][:, g], st["k_own"][b, :lens[b], g]]).double()
                v = torch.cat([st["v_prefix"][:, g], st["v_own"][b, :lens[b], g]]).double()
            for h in range(g * Gq, (g + 1) * Gq):
                a = torch.einsum("td,sd->ts", q[b, :, h], k) * d ** -0.5
                if case["op"] == "prefix":
                    last = case["P"] + lens[b] - T + torch.arange(T, device=a.device)
                    a[torch.arange(a.shape[1], device=a.device)[None] > last.clamp(min=case["P"] - 1)[:, None]] = -math.inf
                y[b, :, h] = torch.einsum("ts,sd->td", torch.softmax(a, -1), v)
    return y
