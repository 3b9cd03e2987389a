"""Cases of the operators that shrink a KV cache: its four-bit form (write, read, attention), the
accumulated attention weight of its tokens, and eviction by that weight.

Four-bit cache (one layer): uint8 [pages][H_kv][b/32][4608].  32 tokens of one head make a strip:
key codes [32][64], value codes [32][64], key scales [32][8], value scales [32][8].  Channel c is the
low (c even) or high (c odd) nibble of code byte c/2: sign, then one of {0, .5, 1, 1.5, 2, 3, 4, 6}.
Scale byte g of a row belongs to channels 16g..16g+15: five exponent bits (bias 15), three mantissa
bits.  A group's scale is the smallest one that is at least max|x|/6; a code is x/scale rounded to the
nearest, ties to the even code.

Where `own` is false, `run` computes each operator in elementary torch operations."""
import math

import torch

own = False

D = 128
STRIP = 32
STRIP_BYTES = 4608
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
SCALE_MAX = 10240.0


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # a decode step of a batch of 8: one token of every sequence goes into its last page
        dict(name="write_token_b8", op="write", B=8, H_q=32, H_kv=8, b=64, lo=32768, hi=65536, paged=True, n=1),
        # a prompt of 32K tokens written at once after prefill
        dict(name="write_prompt_32k", op="write", B=1, H_q=32, H_kv=8, b=64, lo=32768, hi=32768, paged=False, n=32768),
        # a window of 1000 tokens read back for a dense pass over it: ragged lengths, both ends inside a page
        dict(name="read_window_b3", op="read", B=3, H_q=28, H_kv=4, b=128, lo=5000, hi=20000, paged=True, n=1000),
        # a whole layer of 256K tokens read back as bf16 (leaving the four-bit form)
        dict(name="read_layer_256k", op="read", B=1, H_q=28, H_kv=4, b=128, lo=262144, hi=262144, paged=False, n=262144),
        # one decode step over 64 selected blocks of a 32K context, fp32 output
        dict(name="decode_sparse_32k", op="decode", B=1, H_q=32, H_kv=8, b=64, lo=32768, hi=32768, paged=False, M=1,
             n_sel=64, f32=True),
        # the same at 256K with seven heads a group and 128-token blocks
        dict(name="decode_sparse_256k", op="decode", B=1, H_q=28, H_kv=4, b=128, lo=262144, hi=262144, paged=False,
             M=1, n_sel=103, f32=False),
        # three draft tokens checked at once at 512K, five heads a group
        dict(name="decode_draft_512k", op="decode", B=1, H_q=40, H_kv=8, b=64, lo=524288, hi=524288, paged=False, M=3,
             n_sel=32, f32=False),
        # dense attention over every token of a ragged paged batch
        dict(name="decode_dense_b8", op="decode", B=8, H_q=32, H_kv=8, b=64, lo=32768, hi=65536, paged=True, M=1,
             n_sel=0, f32=False),
        # a gated decode step's weights over the 32 selected blocks of a bf16 cache
        dict(name="weights_gate_512k", op="weights", B=1, H_q=40, H_kv=8, b=64, lo=524288, hi=524288, paged=False, M=1,
             n_sel=32, four=False, bias=True),
        # the last 16 tokens' weights over a whole ragged batch, before an eviction
        dict(name="weights_window_b8", op="weights", B=8, H_q=32, H_kv=8, b=64, lo=32768, hi=65536, paged=True, M=16,
             n_sel=0, four=True, bias=False),
        # a batch cut to 4096 tokens a sequence, bf16 pages
        dict(name="evict_b8", op="evict", B=8, H_q=32, H_kv=8, b=64, lo=32768, hi=65536, paged=True, four=False,
             keep=4096, sink=4, recent=128),
        # a 512K context cut to a sixteenth, four-bit pages
        dict(name="evict_512k", op="evict", B=1, H_q=40, H_kv=8, b=64, lo=524288, hi=524288, paged=False, four=True,
             keep=32768, sink=64, recent=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "decode", "decode", "weights", "evict"])
    H_kv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    B = rng.choice([1, 1, 2, 3, 5, 8])
    b = rng.choice([64, 128])
    hi = max(2, min(_log(rng, 2, 262144), 393216 // B))
    lo = rng.choice([hi, max(1, hi // 2), max(1, hi // 7)])
    c = dict(op=op, B=B, H_q=H_kv * G, H_kv=H_kv, b=b, lo=lo, hi=hi, paged=rng.random() < 0.6)
    if op == "write":
        c["n"] = min(_log(rng, 1, 32768), hi, 262144 // (B * H_kv))
    elif op == "read":
        c["n"] = min(_log(rng, 1, 32768), hi, 1048576 // (B * H_kv))
    elif op == "decode":
        n_sel = rng.choice([0, _log(rng, 1, 128)])
        M = rng.choice([1, 1, 1, 2, 3, 4, 8])
        c.update(M=M if n_sel or M * G <= 8 else 1, n_sel=n_sel, f32=rng.random() < 0.4)
    elif op == "weights":
        M = rng.choice([1, 1, 2, 4, 16])
        n_sel = rng.choice([0, _log(rng, 1, 128)])
        four = rng.random() < 0.5
        c.update(M=M if M * G <= 64 else 1, n_sel=n_sel, four=four)
        c["bias"] = bool(c["M"] == 1 and n_sel and not four and rng.random() < 0.6)
    else:
        keep = max(1, min(int(hi * rng.uniform(0.02, 1.1)), 262144 // (B * H_kv)))
        sink = min(keep, rng.choice([0, 4, 33]))
        c.update(four=rng.random() < 0.5, keep=keep, sink=sink, recent=min(keep - sink, rng.choice([0, 1, 16, 130])))
    return c


# ---------------------------------------------------------------------------------------------
# the four-bit form
# ---------------------------------------------------------------------------------------------

def _quantise(x):
    """fp32 [..., 128] -> uint8 codes [..., 64], uint8 scales [..., 8]."""
    g = x.unflatten(-1, (8, 16))
    r = g.abs().amax(-1) / 6
    _, e = torch.frexp(r)                                     # r = m * 2^e, m in [1/2, 1)
    step = torch.ldexp(torch.ones_like(r), torch.clamp(e - 1, min=-14) - 3)
    s = torch.clamp(torch.ceil(r / step) * step, max=SCALE_MAX)
    y = torch.where(s[..., None] > 0, g / torch.where(s > 0, s, 1.0)[..., None], torch.zeros_like(g))
    a = y.abs()
    m = torch.zeros_like(g, dtype=torch.uint8)
    for t, closed in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        m += (a >= t) if closed else (a > t)
    nib = (m | (torch.signbit(g).to(torch.uint8) << 3)).flatten(-2).unflatten(-1, (64, 2))
    scale = (s.to(torch.float16).view(torch.int16) >> 7).to(torch.uint8)
    return nib[..., 0] | (nib[..., 1] << 4), scale


def _strip_parts(x):
    """Key codes, value codes, key scales, value scales of strips [..., 4608] (views)."""
    return (x[..., :2048].unflatten(-1, (32, 64)), x[..., 2048:4096].unflatten(-1, (32, 64)),
            x[..., 4096:4352].unflatten(-1, (32, 8)), x[..., 4352:].unflatten(-1, (32, 8)))


def _values(codes, scales, table):
    """fp32 values [..., 128] of codes [..., 64] and scales [..., 8]."""
    nib = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    s = (scales.to(torch.int16) << 7).view(torch.float16).to(table.dtype)
    return (table[nib].unflatten(-1, (8, 16)) * s[..., None]).flatten(-2)


def _table(device, dtype=torch.float32):
    return torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), dtype=dtype, device=device)


def _blocks(state, pages, which):
    """fp32 keys (0) or values (1) [..., b, 128] of pages [B][H][n] (one head each)."""
    h = torch.arange(state["H_kv"], device=pages.device)[None, :, None]
    if state["four"]:
        parts = _strip_parts(state["kv"][pages, h])
        return _values(parts[which], parts[2 + which], state["table"]).flatten(-3, -2)
    return state["v" if which else "k"][pages, h].float()


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _fill_kv(state, pages, gen, dev):
    """Keys and values ~ N(0,1) times a LogNormal(0, 0.5) scale per head and channel."""
    H, b = state["H_kv"], state["b"]
    sc = torch.exp(0.5 * torch.randn((2, H, 1, D), generator=gen, device=dev))
    if state["four"]:
        state["kv"] = torch.zeros((pages, H, b // STRIP, STRIP_BYTES), dtype=torch.uint8, device=dev)
    else:
        state["k"], state["v"] = (torch.empty((pages, H, b, D), dtype=torch.bfloat16, device=dev) for _ in range(2))
    for p in range(0, pages, 1024):
        n = min(1024, pages - p)
        for i in range(2):
            x = (torch.randn((n, H, b, D), generator=gen, device=dev) * sc[i]).to(torch.bfloat16)
            if state["four"]:
                codes, scales = _quantise(x.float().unflatten(2, (b // STRIP, STRIP)))
                parts = _strip_parts(state["kv"][p:p + n])
                parts[i].copy_(codes)
                parts[2 + i].copy_(scales)
            else:
                state["v" if i else "k"][p:p + n] = x


def _layout(lens, nblk, max_blocks, paged, cpu):
    """A pool of B * max_blocks pages: a seeded permutation of them through a block table, or contiguous pages."""
    B = len(lens)
    if not paged:
        return None, B * max_blocks
    perm = torch.randperm(B * max_blocks, generator=cpu).to(torch.int32)
    bt = torch.full((B, max_blocks), -1, dtype=torch.int32)
    at = 0
    for s in range(B):
        bt[s, :nblk[s]] = perm[at:at + nblk[s]]
        at += nblk[s]
    return bt, B * max_blocks


def _lens(case, seed):
    cpu = torch.Generator().manual_seed(seed * 7919 + 17)
    least = max(case["lo"], case["n"]) if case["op"] == "write" else case["lo"]
    return cpu, torch.randint(least, case["hi"] + 1, (case["B"],), generator=cpu).tolist()


def prepare(case, seed):
    dev = torch.device("cuda")
    cpu, lens = _lens(case, seed)
    gen = torch.Generator(device=dev).manual_seed(seed * 1000003 + 1)
    B, H, b, op = case["B"], case["H_kv"], case["b"], case["op"]
    mb = -(-case["hi"] // b)
    nblk = [-(-x // b) for x in lens]
    bt, pages = _layout(lens, nblk, mb, case["paged"], cpu)
    st = dict(case=case, op=op, B=B, H_kv=H, H_q=case["H_q"], G=case["H_q"] // H, b=b, max_blocks=mb, pages=pages,
              max_len=max(lens), four=case.get("four", True), scale=1.0 / math.sqrt(D), table=_table(dev),
              lens=torch.tensor(lens, dtype=torch.int32, device=dev), bt=None if bt is None else bt.to(dev),
              status=torch.zeros(1, dtype=torch.int32, device=dev))
    bf = lambda *shape: torch.randn(shape, generator=gen, device=dev).to(torch.bfloat16)  # noqa: E731
    if op == "write":
        n = case["n"]
        st["kv"] = torch.zeros((pages, H, b // STRIP, STRIP_BYTES), dtype=torch.uint8, device=dev)
        if n < max(lens):
            _fill_kv(st, pages, gen, dev)
        st["desc"] = torch.zeros((pages, H, 2, D), dtype=torch.bfloat16, device=dev)
        st["k_new"], st["v_new"] = bf(B, n, H, D), bf(B, n, H, D)
        st["pos"] = st["lens"] - n                               # the last n positions
        st["k_out"], st["v_out"] = (torch.zeros((B, n, H, D), dtype=torch.bfloat16, device=dev) for _ in range(2))
        return st
    _fill_kv(st, pages, gen, dev)
    if op == "read":
        n = case["n"]
        st["pos"] = torch.tensor([int(torch.randint(0, max(1, x - n + 1), (1,), generator=cpu)) for x in lens],
                                 dtype=torch.int32, device=dev)
        st["k_out"], st["v_out"] = (torch.zeros((B, n, H, D), dtype=torch.bfloat16, device=dev) for _ in range(2))
        return st
    if op == "evict":
        keep = case["keep"]
        kb = -(-keep // b)
        dbt, dpages = _layout(lens, [kb] * B, kb, case["paged"], cpu)
        st.update(keep=keep, sink=case["sink"], recent=case["recent"], dst_blocks=kb, dst_pages=dpages,
                  dst_bt=None if dbt is None else dbt.to(dev))
        # heavy-tailed weights; a third of the tokens were never attended to (exact ties at 0)
        acc = torch.exp(2 * torch.randn((pages, H, b), generator=gen, device=dev))
        st["acc"] = acc * (torch.rand((pages, H, b), generator=gen, device=dev) > 1 / 3)
        if st["four"]:
            st["dst_kv"] = torch.zeros((dpages, H, b // STRIP, STRIP_BYTES), dtype=torch.uint8, device=dev)
        else:
            st["dst_k"], st["dst_v"] = (torch.zeros((dpages, H, b, D), dtype=torch.bfloat16, device=dev) for _ in range(2))
        st["dst_desc"] = torch.zeros((dpages, H, 2, D), dtype=torch.bfloat16, device=dev)
        st["dst_acc"] = torch.zeros((dpages, H, b), device=dev)
        st["kept"] = torch.full((B, H, keep), -1, dtype=torch.int32, device=dev)
        st["new_lens"] = torch.zeros(B, dtype=torch.int32, device=dev)
        return st
    M = case["M"]
    st["M"] = M
    st["q"] = bf(B, M, case["H_q"], D)
    if case["n_sel"]:
        n_sel = min(case["n_sel"], mb)
        idx = torch.full((B, H, n_sel), -1, dtype=torch.int32)
        cnt = torch.zeros((B, H), dtype=torch.int32)
        for s in range(B):
            k = min(n_sel, nblk[s])
            for h in range(H):  # the last block and k-1 others, ascending
                others = torch.randperm(nblk[s] - 1, generator=cpu)[:k - 1]
                idx[s, h, :k] = torch.cat((others, torch.tensor([nblk[s] - 1]))).sort().values.to(torch.int32)
                cnt[s, h] = k
        st["sel_idx"], st["sel_cnt"] = idx.to(dev), cnt.to(dev)
    else:
        st["sel_idx"] = st["sel_cnt"] = None
    if op == "decode":
        st["out"] = torch.empty((B, M, case["H_q"], D), dtype=torch.float32 if case["f32"] else torch.bfloat16, device=dev)
        st["lse"] = torch.empty((B, M, case["H_q"]), dtype=torch.float32, device=dev)
        return st
    st["bias"] = -torch.rand((B, case["H_q"], n_sel), generator=gen, device=dev) * 8 if case["bias"] else None
    logit, _ = _logits(st)
    st["lse"] = torch.logsumexp(logit.flatten(4), -1).permute(0, 2, 1, 3).reshape(B, M, case["H_q"]).contiguous()
    del logit
    st["acc_in"] = torch.rand((pages, H, b), generator=gen, device=dev)
    st["acc_out"] = st["acc_in"].clone()
    return st


# ---------------------------------------------------------------------------------------------
# the operators' plain forms
# ---------------------------------------------------------------------------------------------

def _pages(state):
    """Pages [B][H][n] of the attended blocks, their logical indices, and which of them count."""
    dev, B, H = state["lens"].device, state["B"], state["H_kv"]
    if state["sel_idx"] is None:
        j = torch.arange(state["max_blocks"], device=dev).expand(B, H, -1)
        live = j * state["b"] < state["lens"][:, None, None]
    else:
        j = state["sel_idx"].long()
        live = torch.arange(j.shape[-1], device=dev) < state["sel_cnt"][..., None]
    j = torch.where(live, j, torch.zeros_like(j))
    s = torch.arange(B, device=dev)[:, None, None]
    pages = state["bt"].long()[s, j] if state["bt"] is not None else s * state["max_blocks"] + j
    return torch.where(live, pages, torch.zeros_like(pages)), j, live


def _logits(state):
    """fp32 logits [B][H][M][G][n][b] of the attended blocks (-inf where masked), and their pages."""
    B, H, M, G, b = state["B"], state["H_kv"], state["M"], state["G"], state["b"]
    pages, j, live = _pages(state)
    k = _blocks(state, pages, 0)
    q = state["q"].float().view(B, M, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, M * G, D)
    x = torch.matmul(q, k.flatten(2, 3).transpose(-1, -2)).view(B, H, M, G, -1, b) * state["scale"]
    if state.get("bias") is not None:
        x += state["bias"].view(B, 1, H, G, -1).transpose(1, 2)[..., None]
    tok = j[..., None] * b + torch.arange(b, device=k.device)
    limit = state["lens"][:, None] - M + 1 + torch.arange(M, device=k.device)          # [B][M]
    see = live[..., None][:, :, None] & (tok[:, :, None] < limit[:, None, :, None, None])
    return torch.where(see[:, :, :, None], x, -math.inf), pages


def _decode(state):
    B, H, M, G = state["B"], state["H_kv"], state["M"], state["G"]
    x, pages = _logits(state)
    x = x.flatten(4)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m > -math.inf, m, 0.0))
    z = p.sum(-1, keepdim=True)
    v = _blocks(state, pages, 1).flatten(2, 3)
    o = torch.matmul((p / torch.where(z > 0, z, 1.0)).flatten(2, 3), v).view(B, H, M, G, D)
    lse = torch.where(z > 0, m + torch.log(z), -math.inf)[..., 0]
    return (o.permute(0, 2, 1, 3, 4).reshape(B, M, H * G, D).to(state["out"].dtype),
            lse.permute(0, 2, 1, 3).reshape(B, M, H * G))


def _weights(state):
    B, H, M, G, b = state["B"], state["H_kv"], state["M"], state["G"], state["b"]
    x, pages = _logits(state)
    lse = state["lse"].view(B, M, H, G).permute(0, 2, 1, 3)[..., None, None]
    w = torch.where(lse > -math.inf, torch.exp(x - lse), 0.0).sum((2, 3))               # [B][H][n][b]
    _, j, live = _pages(state)
    inside = live[..., None] & (j[..., None] * b + torch.arange(b, device=w.device) < state["lens"][:, None, None, None])
    at = inside.nonzero(as_tuple=True)
    page, head = pages[at[:3]], at[1]
    state["acc_out"][page, head, at[3]] = state["acc_in"][page, head, at[3]] + w[at]
    return state["acc_out"]


def _rows(state, pos, n):
    """Page and row of positions pos..pos+n-1 of every sequence, and which are below its length."""
    t = pos.long()[:, None] + torch.arange(n, device=pos.device)
    inside = t < state["lens"][:, None]
    j = torch.clamp(t // state["b"], max=state["max_blocks"] - 1)
    s = torch.arange(state["B"], device=pos.device)[:, None]
    pages = state["bt"].long()[s, j] if state["bt"] is not None else s * state["max_blocks"] + j
    return torch.where(inside, pages, torch.zeros_like(pages)), t % state["b"], inside, j


def _read(state, n):
    pages, row, inside, _ = _rows(state, state["pos"], n)
    x = state["kv"].permute(0, 2, 1, 3)[pages, row // STRIP]                            # [B][n][H][4608]
    parts = _strip_parts_at(x, row % STRIP)
    k = _values(parts[0], parts[2], state["table"]).to(torch.bfloat16)
    v = _values(parts[1], parts[3], state["table"]).to(torch.bfloat16)
    keep = inside[..., None, None]
    return torch.where(keep, k, state["k_out"]), torch.where(keep, v, state["v_out"])


def _strip_parts_at(x, r):
    """Row r [B][n] of strips x [B][n][H][4608]."""
    idx = r[:, :, None, None]
    take = lambda base, width: torch.gather(x, 3, (base + idx * width + torch.arange(width, device=x.device)).expand(*x.shape[:3], width))  # noqa: E731
    return take(0, 64), take(2048, 64), take(4096, 8), take(4352, 8)


def _write(state):
    n, H, b = state["k_new"].shape[1], state["H_kv"], state["b"]
    pages, row, _, j = _rows(state, state["pos"], n)
    h = torch.arange(H, device=pages.device)
    page, strip, r = pages[..., None], (row // STRIP)[..., None], (row % STRIP)[..., None]
    parts = _strip_parts(state["kv"])
    for i, x in enumerate((state["k_new"], state["v_new"])):
        codes, scales = _quantise(x.float())
        parts[i][page, h, strip, r] = codes
        parts[2 + i][page, h, strip, r] = scales
    # descriptors of the touched blocks from all of their valid keys
    first, last = state["pos"].long() // b, (state["pos"].long() + n - 1) // b
    jt = first[:, None] + torch.arange((n - 1) // b + 2, device=pages.device)
    hit = (jt <= last[:, None]) & (jt * b < state["lens"][:, None])
    s, c = hit.nonzero(as_tuple=True)
    jj = jt[s, c]
    pg = state["bt"].long()[s, jj] if state["bt"] is not None else s * state["max_blocks"] + jj
    kp = _strip_parts(state["kv"][pg])
    k = _values(kp[0], kp[2], state["table"]).flatten(2, 3)                             # [hits][H][b][128]
    ok = (jj[:, None] * b + torch.arange(b, device=pages.device) < state["lens"][s][:, None])[:, None, :, None]
    state["desc"][pg, :, 0] = torch.where(ok, k, math.inf).amin(2).to(torch.bfloat16)
    state["desc"][pg, :, 1] = torch.where(ok, k, -math.inf).amax(2).to(torch.bfloat16)
    return state["desc"]


def _evict(state):
    B, H, b, keep = state["B"], state["H_kv"], state["b"], state["keep"]
    dev, lens = state["lens"].device, state["lens"].long()
    s = torch.arange(B, device=dev)[:, None, None]
    h = torch.arange(H, device=dev)[None, :, None]
    t = torch.arange(state["max_blocks"] * b, device=dev)

    def page_of(table, blocks, tok):
        jb = torch.clamp(tok // b, max=blocks - 1)
        pg = table.long()[s, jb] if table is not None else s * blocks + jb
        return pg

    inside = (t < lens[:, None])[:, None].expand(B, H, -1)
    pg = torch.where(inside, page_of(state["bt"], state["max_blocks"], t.expand(B, H, -1)), 0)
    w = state["acc"][pg, h, (t % b).expand(B, H, -1)]
    forced = (t < state["sink"]) | (t >= lens[:, None] - state["recent"])[:, None]
    w = torch.where(forced, math.inf, w)
    w = torch.where(inside, w, -math.inf)
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :keep].sort(-1).values
    new = torch.clamp(lens, max=keep)
    live = torch.arange(keep, device=dev) < new[:, None, None]
    live = live.expand(B, H, -1)
    if order.shape[-1] < keep:
        order = torch.nn.functional.pad(order, (0, keep - order.shape[-1]))
    src = torch.where(live, order, 0)
    to = torch.arange(keep, device=dev).expand(B, H, -1)
    sp, dp = page_of(state["bt"], state["max_blocks"], src), page_of(state["dst_bt"], state["dst_blocks"], to)
    at = live.nonzero(as_tuple=True)
    sp, sr, dp, dr, hh = sp[at], src[at] % b, dp[at], at[2] % b, at[1]
    if state["four"]:
        for x, y in zip(_strip_parts(state["kv"]), _strip_parts(state["dst_kv"])):
            y[dp, hh, dr // STRIP, dr % STRIP] = x[sp, hh, sr // STRIP, sr % STRIP]
        parts = _strip_parts(state["kv"])
        k = _values(parts[0][sp, hh, sr // STRIP, sr % STRIP], parts[2][sp, hh, sr // STRIP, sr % STRIP], state["table"])
    else:
        state["dst_k"][dp, hh, dr] = state["k"][sp, hh, sr]
        state["dst_v"][dp, hh, dr] = state["v"][sp, hh, sr]
        k = state["k"][sp, hh, sr].float()
    state["dst_acc"][dp, hh, dr] = state["acc"][sp, hh, sr]
    state["kept"][at] = src[at].to(torch.int32)
    state["new_lens"].copy_(new)
    cell = (dp * H + hh)[:, None].expand(-1, D)
    for i, (start, how) in enumerate(((math.inf, "amin"), (-math.inf, "amax"))):
        x = torch.full((state["dst_pages"] * H, D), start, device=dev).scatter_reduce(0, cell, k, how)
        x = x.view(-1, H, D)
        state["dst_desc"][:, :, i] = torch.where(x.abs() < math.inf, x.to(torch.bfloat16), state["dst_desc"][:, :, i])
    return _evicted(state)


def _evicted(state):
    moved = {"kv": state["dst_kv"]} if state["four"] else {"k": state["dst_k"], "v": state["dst_v"]}
    return {**moved, "desc": state["dst_desc"], "acc": state["dst_acc"], "kept": state["kept"], "lens": state["new_lens"]}


# ---------------------------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------------------------

def _handles(state):
    """The caches of the layer (and buffers) as a program keeps them from step to step."""
    if "handles" not in state:
        from block_sparse_gqa_min_b200 import sba

        common = dict(seq_lens=state["lens"], H_q=state["H_q"], max_blocks=state["max_blocks"], max_len=state["max_len"],
                      block_table=state["bt"], status=state["status"])
        got = {"sba": sba}
        if state["four"]:
            got["c"] = sba.Cache4(kv=state["kv"], desc=state.get("desc"), **common)
        else:
            got["c"] = sba.Cache(k=state["k"], v=state["v"], **common)
        if state["op"] == "decode":
            n_max = 0 if state["sel_idx"] is None else state["sel_idx"].shape[-1]
            size = sba.sba_decode_kv4_workspace_size(got["c"], state["M"], n_max)
            got["ws"] = torch.zeros(max(16, size), dtype=torch.uint8, device=state["lens"].device)
        if state["op"] == "evict":
            to = dict(seq_lens=state["new_lens"], H_q=state["H_q"], max_blocks=state["dst_blocks"], max_len=state["keep"],
                      block_table=state["dst_bt"], desc=state["dst_desc"], status=state["status"])
            got["dst"] = (sba.Cache4(kv=state["dst_kv"], **to) if state["four"]
                          else sba.Cache(k=state["dst_k"], v=state["dst_v"], **to))
            got["p"] = sba.evict_params(state["keep"], state["sink"], state["recent"])
        state["handles"] = got
    return state["handles"]


def run(state):
    op = state["op"]
    if not own:
        if op == "write":
            desc = _write(state)
            k, v = _read(state, state["k_new"].shape[1])
            return {"k": k, "v": v, "desc": desc}
        if op == "read":
            return _read(state, state["k_out"].shape[1])
        return {"decode": _decode, "weights": _weights, "evict": _evict}[op](state)
    got = _handles(state)
    sba, c = got["sba"], got["c"]
    if op == "write":
        sba.sba_append_kv4(c, state["k_new"], state["v_new"], state["pos"])
        sba.sba_read_kv4(c, state["pos"], state["k_out"], state["v_out"])
        return {"k": state["k_out"], "v": state["v_out"], "desc": state["desc"]}
    if op == "read":
        sba.sba_read_kv4(c, state["pos"], state["k_out"], state["v_out"])
        return state["k_out"], state["v_out"]
    if op == "decode":
        sba.sba_decode_kv4(c, state["q"], state["scale"], state["out"], got["ws"], lse_out=state["lse"],
                           sel_idx=state["sel_idx"], sel_cnt=state["sel_cnt"])
        return state["out"], state["lse"]
    if op == "weights":
        if state["four"]:
            sba.sba_accumulate_weights_kv4(c, state["q"], state["lse"], state["scale"], state["acc_in"],
                                           state["acc_out"], sel_idx=state["sel_idx"], sel_cnt=state["sel_cnt"])
        else:
            sba.sba_accumulate_weights(c, state["q"], state["lse"], state["scale"], state["acc_in"], state["acc_out"],
                                       sel_idx=state["sel_idx"], sel_cnt=state["sel_cnt"], gate_bias=state["bias"])
        return state["acc_out"]
    evict = sba.sba_evict_kv4 if state["four"] else sba.sba_evict
    evict(c, state["acc"], got["p"], got["dst"], state["new_lens"], state["kept"], acc_dst=state["dst_acc"])
    return _evicted(state)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------

def _attended(case):
    """Tokens that a pass attends to (over the batch, per KV head), at the mean length."""
    mean = (case["lo"] + case["hi"]) / 2
    if not case["n_sel"]:
        return case["B"] * mean
    return case["B"] * min(case["n_sel"] * case["b"], mean)


def work(case):
    B, H, Hq, op = case["B"], case["H_kv"], case["H_q"], case["op"]
    if op in ("write", "read"):
        rows = B * min(case["n"], case["hi"]) * H
        bytes_ = rows * (144 + 512)                       # codes and scales read, bf16 rows written
        if op == "write":
            bytes_ += rows * (512 + 144) + (B * H * 512 * (-(-case["n"] // case["b"])))
        return {"bytes": bytes_, "flops": 0}
    if op == "evict":
        mean = (case["lo"] + case["hi"]) / 2
        kept = B * min(case["keep"], mean) * H
        row = 144 if case["four"] else 512
        return {"bytes": 4 * B * mean * H + kept * (2 * row + 4 + 4) + kept / case["b"] * 512, "flops": 0}
    M, n = case["M"], _attended(case)
    if op == "decode":
        q = B * M * Hq * D
        return {"bytes": n * H * 144 + q * 2 + q * (4 if case["f32"] else 2), "flops": 4 * n * M * Hq * D}
    row = 72 if case["four"] else 256
    return {"bytes": n * H * (row + 8) + B * M * Hq * (D * 2 + 4), "flops": 2 * n * M * Hq * D}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits, sequence by sequence
# ---------------------------------------------------------------------------------------------

def _grid64(x):
    """bf16 [..., 128] -> the value each element has in the four-bit form, by searching the grid of scales and codes."""
    dev = x.device
    g = x.double().unflatten(-1, (8, 16))
    byte = torch.arange(227, device=dev, dtype=torch.float64)                           # scales 0 .. 10240
    e, m = torch.floor(byte / 8), byte % 8
    scales = torch.where(e > 0, 2.0 ** (e - 15) * (1 + m / 8), 2.0 ** -14 * m / 8)
    at = torch.clamp(torch.searchsorted(6 * scales, g.abs().amax(-1).contiguous()), max=226)
    s = scales[at][..., None]
    grid = torch.tensor(MAGNITUDES, dtype=torch.float64, device=dev)
    hi = torch.clamp(torch.searchsorted(grid, (g.abs() / torch.where(s > 0, s, 1.0)).contiguous()), max=7)
    lo = torch.clamp(hi - 1, min=0)
    d_hi, d_lo = (grid[hi] * s - g.abs()).abs(), (g.abs() - grid[lo] * s).abs()
    code = torch.where((d_lo < d_hi) | ((d_lo == d_hi) & (lo % 2 == 0)), lo, hi)
    return (torch.sign(g) * grid[code] * s).flatten(-2)


def _seq64(st, s, which):
    """All keys (0) or values (1) of sequence s in 64 bits: [H][len][128]."""
    n, b = int(st["lens"][s]), st["b"]
    blocks = -(-n // b)
    pages = st["bt"][s, :blocks].long() if st["bt"] is not None else s * st["max_blocks"] + torch.arange(blocks, device=st["lens"].device)
    if not st["four"]:
        x = st["v" if which else "k"][pages].double()                                   # [blocks][H][b][128]
    else:
        raw = st["kv"][pages]
        codes = raw[..., 2048 * which:2048 * which + 2048].reshape(*raw.shape[:3], 32, 64).int()
        sc = raw[..., 4096 + 256 * which:4352 + 256 * which].reshape(*raw.shape[:3], 32, 8).int()
        e, m = sc // 8, (sc % 8).double() / 8
        scale = torch.where(e > 0, torch.ldexp(1 + m, e - 15), torch.ldexp(m, torch.full_like(e, -14)))
        nib = torch.stack((codes % 16, codes // 16), -1).flatten(-2)
        mag = torch.tensor(MAGNITUDES, dtype=torch.float64, device=raw.device)[nib % 8]
        x = torch.where(nib >= 8, -mag, mag) * scale.repeat_interleave(16, -1)
        x = x.flatten(2, 3)
    return x.transpose(0, 1).flatten(1, 2)[:, :n]


def _row_logits64(st, s, h, keys):
    """Logits [M*G][tokens] of sequence s, head h in 64 bits over the tokens it attends to, and those tokens."""
    n, M, G, b = int(st["lens"][s]), st["M"], st["G"], st["b"]
    dev = keys.device
    if st["sel_idx"] is None:
        tok = torch.arange(n, device=dev)
        pos = None
    else:
        sel = st["sel_idx"][s, h, :int(st["sel_cnt"][s, h])].long()
        tok = (sel[:, None] * b + torch.arange(b, device=dev)).flatten()
        pos = torch.arange(sel.numel(), device=dev).repeat_interleave(b)[tok < n]
        tok = tok[tok < n]
    q = st["q"][s, :, h * G:(h + 1) * G].double()                                       # [M][G][128]
    x = torch.einsum("mgd,td->mgt", q, keys[h][tok]) / math.sqrt(D)
    if st.get("bias") is not None:
        x = x + st["bias"][s, h * G:(h + 1) * G].double()[:, pos]
    last = n - M + torch.arange(M, device=dev)                                          # the last position a row sees
    return x.masked_fill(tok > last[:, None, None], -math.inf), tok


def exact(case, seed):
    st = prepare(case, seed)
    op, B, H = case["op"], case["B"], case["H_kv"]
    if op == "read":
        k, v = (torch.zeros(st["k_out"].shape, dtype=torch.float64, device=st["lens"].device) for _ in range(2))
        for s in range(B):
            a = int(st["pos"][s])
            for which, out in ((0, k), (1, v)):
                x = _seq64(st, s, which)[:, a:a + case["n"]].transpose(0, 1)
                out[s, :x.shape[0]] = x
        return k, v
    if op == "write":
        k, v = _grid64(st["k_new"]), _grid64(st["v_new"])
        desc = st["desc"].double()
        for s in range(B):
            a, n, b = int(st["pos"][s]), int(st["lens"][s]), st["b"]
            keys = _seq64(st, s, 0).clone()
            keys[:, a:a + case["n"]] = k[s].transpose(0, 1)[:, :n - a]
            for j in range(a // b, -(-n // b)):
                page = int(st["bt"][s, j]) if st["bt"] is not None else s * st["max_blocks"] + j
                desc[page, :, 0] = keys[:, j * b:(j + 1) * b].amin(1)
                desc[page, :, 1] = keys[:, j * b:(j + 1) * b].amax(1)
        return {"k": k, "v": v, "desc": desc}
    if op == "decode":
        M, G = st["M"], st["G"]
        out = torch.zeros((B, M, H * G, D), dtype=torch.float64, device=st["lens"].device)
        lse = torch.full((B, M, H * G), -math.inf, dtype=torch.float64, device=out.device)
        for s in range(B):
            keys, vals = _seq64(st, s, 0), _seq64(st, s, 1)
            for h in range(H):
                x, tok = _row_logits64(st, s, h, keys)
                z = torch.logsumexp(x, -1)
                p = torch.where(z[..., None] > -math.inf, torch.exp(x - z[..., None]), 0.0)
                out[s, :, h * G:(h + 1) * G] = torch.einsum("mgt,td->mgd", p, vals[h][tok])
                lse[s, :, h * G:(h + 1) * G] = z
        return out, lse
    if op == "weights":
        G, b = st["G"], st["b"]
        acc = st["acc_out"].double()
        for s in range(B):
            keys = _seq64(st, s, 0)
            for h in range(H):
                x, tok = _row_logits64(st, s, h, keys)
                z = st["lse"][s, :, h * G:(h + 1) * G].double()[..., None]
                w = torch.where(z > -math.inf, torch.exp(x - z), 0.0).sum((0, 1))
                j = tok // b
                page = st["bt"][s].long()[j] if st["bt"] is not None else s * st["max_blocks"] + j
                acc[page, h, tok % b] = st["acc_in"][page, h, tok % b].double() + w
        return acc
    return None                                       # eviction moves rows (bytes) and picks by its input: nothing is computed
