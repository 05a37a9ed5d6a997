"""The 8-bit paged K/V cache: what its operators compute, and the calls that are timed.

A cache is a pool of pages.  ``k_pages`` and ``v_pages`` are [P, Hkv, ps, d] in an
8-bit floating type, ``k_scale`` and ``v_scale`` [P, Hkv] float32: the element that
code c stands for is c * scale[page, head].  ``table`` [B, T] int32 lists each
sequence's pages: slot t of sequence b lives in page table[b, t // ps], row t % ps.
Three operators work on it:

  attend  O = softmax(s * Q K^T) V of few queries a sequence over its ``lens[b]`` slots,
          grouped query heads, with the log-sum-exp of each row and, where asked for,
          each slot's attention weight, summed over the query rows that share the
          head, added into an accumulator
  append  new keys and values, quantised with one power-of-two scale a page and head,
          behind the slots that are there
  evict   the slots with the smallest accumulated weight leave (the latest tokens
          stay): kept slots behind the new length move into the holes before it

``own`` false: their plain forms in torch; ``own`` true: the library's kernels.
"""
import math

import torch

own = False

FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FP8_MAX = {"e4m3": 448.0, "e5m2": 57344.0}
DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------- cases
def _attend(name, B, Hq, Hkv, Nq, d, length, ps, dtype="bf16", cache="e4m3", ragged=False, weights=False):
    return dict(name=name, op="attend", B=B, Hq=Hq, Hkv=Hkv, Nq=Nq, d=d, len=length, ps=ps, dtype=dtype, cache=cache,
                ragged=ragged, weights=weights, N=0, keep=0, recent=0)


def _append(name, B, Hkv, N, d, length, ps, dtype="bf16", cache="e4m3", ragged=False):
    return dict(name=name, op="append", B=B, Hq=Hkv, Hkv=Hkv, Nq=1, d=d, len=length, ps=ps, dtype=dtype, cache=cache,
                ragged=ragged, weights=False, N=N, keep=0, recent=0)


def _evict(name, B, Hkv, d, length, keep, recent, ps, cache="e4m3", ragged=False):
    return dict(name=name, op="evict", B=B, Hq=Hkv, Hkv=Hkv, Nq=1, d=d, len=length, ps=ps, dtype="bf16", cache=cache,
                ragged=ragged, weights=False, N=0, keep=keep, recent=recent)


def listed():
    return [
        # the smallest call: one request at the start of its answer, a few hundred tokens
        _attend("attend_short", 1, 8, 2, 1, 64, 257, 16),
        # an ordinary batch being served: requests of very different lengths, one just begun, one empty
        _attend("attend_ragged", 24, 32, 8, 1, 128, 5000, 64, ragged=True),
        # one long document, one question: the long axis is all there is to split
        _attend("attend_document", 1, 32, 8, 1, 128, 131071, 64),
        # every query head with keys of its own, 32K keys: the most bytes
        _attend("attend_all_heads", 4, 32, 32, 1, 128, 32768, 128),
        # five drafted tokens verified at once, wide heads, the other types
        _attend("attend_drafted", 8, 16, 2, 5, 256, 8191, 32, "fp16", "e5m2"),
        # a batch that keeps count of where its attention goes, for eviction
        _attend("attend_weights", 16, 32, 8, 1, 128, 8192, 64, weights=True),
        # one token for each of 64 requests
        _append("append_token", 64, 8, 1, 128, 4096, 64, ragged=True),
        # four prompts behind a shared beginning
        _append("append_prompt", 4, 8, 8192, 128, 100, 64),
        # prompts of different lengths in one padded batch, narrow heads, the other types
        _append("append_padded", 12, 4, 1500, 64, 333, 16, "fp16", "e5m2", ragged=True),
        # a budget of 2048 slots kept while decoding: 32 tokens leave
        _evict("evict_steady", 32, 8, 128, 2080, 2048, 256, 64),
        # long prompts cut to a quarter
        _evict("evict_prompt", 8, 8, 128, 16384, 4096, 512, 64),
        # one decoding step of a batch: the new token's key and value, then its attention with the count of weights
        dict(_attend("step", 32, 32, 8, 1, 128, 3001, 64, ragged=True, weights=True), op="step", N=1),
    ]


def draw(rng):
    """Another case of the ranges above: log-uniform sizes, both types of each, every page size and head width."""
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["attend", "attend", "attend", "append", "evict", "step"])
    d, ps = rng.choice([64, 128, 128, 256]), rng.choice([16, 32, 64, 128])
    dtype, cache = rng.choice(["bf16", "bf16", "fp16"]), rng.choice(["e4m3", "e4m3", "e5m2"])
    hkv = rng.choice([1, 2, 4, 8, 8, 3])
    ragged = rng.random() < 0.5
    budget = 1 << 28  # bytes of keys: a quarter of the largest listed case
    if op == "append":
        B, N = log(1, 64), log(1, 6000)
        length = log(1, 4000)
        N = max(1, min(N, budget // 2 // (B * hkv * d)))
        length = max(1, min(length, budget // (B * hkv * d)))
        return {k: v for k, v in _append("", B, hkv, N, d, length, ps, dtype, cache, ragged).items() if k != "name"}
    length = log(100, 100000)
    B = max(1, min(log(1, 64), budget // (length * hkv * d)))
    length = min(length, budget // (B * hkv * d))
    if op == "evict":
        keep = max(1, int(length * rng.uniform(0.1, 1.0)))
        recent = int(keep * rng.uniform(0.0, 0.9))
        return {k: v for k, v in _evict("", B, hkv, d, length, keep, recent, ps, cache, ragged).items() if k != "name"}
    group, nq = rng.choice([1, 2, 4, 4, 7, 8]), 1 if op == "step" else rng.choice([1, 1, 1, 2, 3, 4, 6])
    weights = op == "step" or rng.random() < 0.3
    c = _attend("", B, hkv * group, hkv, nq, d, length, ps, dtype, cache, ragged, weights)
    c.update(op=op, N=1 if op == "step" else 0)
    return {k: v for k, v in c.items() if k != "name"}


def _lens(case):
    """Slots filled before the call.  Ragged: spread over [0, len], one full, one of a single slot, one empty."""
    B, n = case["B"], case["len"]
    if not case["ragged"]:
        return [n] * B
    got = [int(n * ((0.618034 * b + 0.37) % 1.0)) for b in range(B)]
    got[0] = n
    if B > 2:
        got[1] = min(1, n)
    if B > 3:
        got[2] = 0
    return got


def _counts(case):
    """Tokens that each sequence appends: of a padded batch, fewer than N for most, none for one."""
    B, N = case["B"], case["N"]
    if not case["ragged"] or N == 1:
        return [N] * B
    got = [max(1, int(N * ((0.618034 * b + 0.61) % 1.0))) for b in range(B)]
    got[0] = N
    if B > 3:
        got[3] = 0
    return got


# ---------------------------------------------------------------- inputs
def _quantised_pool(g, dev, P, case):
    """Codes and scales of P pages: normal values with a few channels that are larger, as keys have them."""
    hkv, ps, d, kind = case["Hkv"], case["ps"], case["d"], case["cache"]
    channel = torch.exp(0.6 * torch.randn(1, hkv, 1, d, generator=g, device=dev))
    x = torch.randn(P, hkv, ps, d, generator=g, device=dev, dtype=torch.bfloat16) * channel.to(torch.bfloat16)
    scale = x.abs().amax((2, 3)).float() / FP8_MAX[kind]
    codes = (x.float() / scale[..., None, None]).clamp_(-FP8_MAX[kind], FP8_MAX[kind]).to(FP8[kind])
    return codes.contiguous(), scale.contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    B, hkv, hq, nq, d, ps = (case[k] for k in ("B", "Hkv", "Hq", "Nq", "d", "ps"))
    T = (case["len"] + case["N"]) // ps + 2  # a table has room for what comes next
    P = B * T + 3                            # a pool has pages of others and free ones
    state = {"case": dict(case)}
    state["table"] = torch.randperm(P, generator=g, device=dev)[:B * T].view(B, T).to(torch.int32)
    state["k_pages"], state["k_scale"] = _quantised_pool(g, dev, P, case)
    state["v_pages"], state["v_scale"] = _quantised_pool(g, dev, P, case)
    state["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device=dev)
    state["new_lens"] = torch.zeros_like(state["lens"])
    dt = DTYPE[case["dtype"]]
    if case["op"] in ("attend", "step"):
        state["q"] = torch.randn(B, hq, nq, d, generator=g, device=dev).mul_(1.5).to(dt)
        state["o"] = torch.zeros(B, hq, nq, d, device=dev, dtype=dt)
        state["lse"] = torch.zeros(B, hq, nq, device=dev)
    if case["op"] in ("append", "step"):
        state["k"] = torch.randn(B, hkv, case["N"], d, generator=g, device=dev).to(dt)
        state["v"] = torch.randn(B, hkv, case["N"], d, generator=g, device=dev).to(dt)
        state["counts"] = torch.tensor(_counts(case), dtype=torch.int32, device=dev)
    if case["weights"] or case["op"] == "evict":
        # weights as attention leaves them: a few slots take most of it
        state["acc"] = torch.exp(1.5 * torch.randn(B, hkv, T * ps, generator=g, device=dev))
    if case["op"] == "evict":
        # slots are in the order of their tokens; earlier evictions left gaps between the positions
        step = torch.randint(1, 4, (B, hkv, T * ps), generator=g, device=dev, dtype=torch.int32)
        state["positions"] = torch.cumsum(step, 2).to(torch.int32)
        state["acc_now"], state["positions_now"] = state["acc"].clone(), state["positions"].clone()
    return state


# ---------------------------------------------------------------- plain forms
def _rows(pages, table):
    """The sequences' slots in order, [B, Hkv, T * ps, d], as the codes' values."""
    x = pages.view(torch.uint8)[table.long()].view(pages.dtype).float()
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _slot_scales(scale, table, ps):
    return scale[table.long()].permute(0, 2, 1).repeat_interleave(ps, 2)


def _plain_attend(state, lens):
    case = state["case"]
    B, hkv, hq, nq, d, ps = (case[k] for k in ("B", "Hkv", "Hq", "Nq", "d", "ps"))
    table, q = state["table"], state["q"].float().view(B, hkv, hq // hkv * nq, d)
    k = _rows(state["k_pages"], table) * _slot_scales(state["k_scale"], table, ps)[..., None]
    s = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    del k
    slot = torch.arange(s.shape[3], device=s.device)
    # query i is the token at slot lens - Nq + i: it sees the slots up to its own
    last = lens.long()[:, None] - nq + torch.arange(nq, device=s.device)
    seen = (slot <= last[..., None]).repeat(1, hq // hkv, 1)[:, None]
    s = s.masked_fill(~seen, -math.inf)
    m = s.amax(3, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(s - m)
    l = p.sum(3, keepdim=True)
    v = _rows(state["v_pages"], table) * _slot_scales(state["v_scale"], table, ps)[..., None]
    o = torch.matmul(p, v) / torch.where(l > 0, l, torch.ones_like(l))
    state["o"].copy_(o.view(B, hq, nq, d))
    state["lse"].copy_((m + torch.log(l)).view(B, hq, nq))
    if case["weights"]:
        state["acc"] += (p / torch.where(l > 0, l, torch.ones_like(l))).sum(2)


def _power_of_two(amax, kind):
    """The smallest power of two s, at least 2^-100, with amax <= (largest code) * s (that code is 7/8 of a power of two)."""
    mant, expo = torch.frexp(amax)
    e = expo - (9 if kind == "e4m3" else 16) + (mant > 0.875).int()
    e = torch.where(amax > 0, e, torch.full_like(e, -100)).clamp(min=-100)
    return ((e + 127) << 23).view(torch.float32)  # the power itself: pow() need not be exact


def _plain_append_one(pages, scale, x, state, lens, counts):
    case = state["case"]
    hkv, d, ps, N, kind = (case[k] for k in ("Hkv", "d", "ps", "N", "cache"))
    touched = (N - 1) // ps + 2  # pages that N tokens can reach
    first = lens.long() // ps
    local = first[:, None] + torch.arange(touched, device=x.device)
    page = state["table"].long().gather(1, local)  # [B, touched]
    slot = (local[..., None] * ps + torch.arange(ps, device=x.device)).flatten(1)
    token = slot - lens.long()[:, None]
    new = (token >= 0) & (token < counts.long()[:, None])
    B = slot.shape[0]
    at = token.clamp(0, N - 1)[:, None, :, None].expand(-1, hkv, -1, d)
    val = x.float().gather(2, at).view(B, hkv, touched, ps, d)
    new = new.view(B, 1, touched, ps).expand(-1, hkv, -1, -1)
    old = (token < 0).view(B, 1, touched, ps).expand(-1, hkv, -1, -1)
    amax = (val.abs() * new[..., None]).amax((3, 4))
    need = _power_of_two(amax, kind)
    was = scale[page].transpose(1, 2)  # [B, hkv, touched]
    now = torch.where(old.any(3), torch.maximum(was, need), need)
    now = torch.where(new.any(3), now, was)
    codes = pages.view(torch.uint8)[page].permute(0, 2, 1, 3, 4)  # [B, hkv, touched, ps, d]
    fresh = (val / now[..., None, None] * new[..., None]).to(pages.dtype).view(torch.uint8)
    kept = (codes.contiguous().view(pages.dtype).float() * (was / now)[..., None, None]).to(pages.dtype).view(torch.uint8)
    codes = torch.where(new[..., None], fresh, torch.where(old[..., None], kept, codes))
    pages.view(torch.uint8)[page] = codes.permute(0, 2, 1, 3, 4)
    scale[page] = now.transpose(1, 2)


def _plain_append(state):
    lens, counts = state["lens"], state["counts"]
    _plain_append_one(state["k_pages"], state["k_scale"], state["k"], state, lens, counts)
    _plain_append_one(state["v_pages"], state["v_scale"], state["v"], state, lens, counts)
    state["new_lens"].copy_(lens + counts)
    if "acc" in state:  # new slots start without weight
        token = torch.arange(state["acc"].shape[2], device=lens.device) - lens.long()[:, None]
        new = (token >= 0) & (token < counts.long()[:, None])
        state["acc"].masked_fill_(new[:, None], 0.0)


def _plain_evict_one(pages, scale, state, src, valid, dest_pages, width):
    """Rows src [B, Hkv, width * ps] into the first pages of each sequence, at the largest scale that meets there."""
    hkv, ps, d = (state["case"][k] for k in ("Hkv", "ps", "d"))
    B = src.shape[0]
    head = torch.arange(hkv, device=src.device)[None, :, None]
    src_page = state["table"].long()[:, None].expand(-1, hkv, -1).gather(2, src // ps)
    rows = pages.view(torch.uint8).view(-1, d)[(src_page * hkv + head) * ps + src % ps]
    s_src = scale[src_page, head]
    own_scale = scale[dest_pages].transpose(1, 2)  # [B, hkv, width]
    s_new = torch.where(valid, s_src, torch.zeros_like(s_src)).view(B, hkv, width, ps).amax(3)
    any_valid = valid.view(B, -1, width, ps).any(3)
    s_new = torch.where(any_valid, s_new, own_scale)
    ratio = s_src / s_new.repeat_interleave(ps, 2)
    moved = (rows.view(pages.dtype).float() * ratio[..., None]).to(pages.dtype).view(torch.uint8)
    rows = torch.where(valid[..., None], moved, rows)
    pages.view(torch.uint8)[dest_pages] = rows.view(B, hkv, width, ps, d).transpose(1, 2)
    scale[dest_pages] = s_new.transpose(1, 2)


def _plain_evict(state):
    case = state["case"]
    hkv, ps, keep, recent = (case[k] for k in ("Hkv", "ps", "keep", "recent"))
    acc, pos, lens = state["acc"], state["positions"], state["lens"].long()
    acc.copy_(state["acc_now"])
    pos.copy_(state["positions_now"])
    B, _, L = acc.shape
    slot = torch.arange(L, device=acc.device).expand(B, hkv, L)
    n, m = lens[:, None, None], lens.clamp(max=keep)[:, None, None]
    filled = slot < n
    latest = torch.where(filled, pos, torch.full_like(pos, -1)).amax(2, keepdim=True)
    protected = filled & (pos > latest - recent)
    rank_by = torch.where(protected, torch.full_like(acc, math.inf), acc)
    rank_by = torch.where(filled, rank_by, torch.full_like(acc, -math.inf))
    order = torch.sort(rank_by, dim=2, descending=True, stable=True)[1]
    kept = torch.zeros(B, hkv, L, dtype=torch.bool, device=acc.device).scatter_(2, order, (slot < m))
    hole, mover = ~kept & (slot < m), kept & (slot >= m)
    mover_of = torch.zeros(B, hkv, L + 1, dtype=torch.long, device=acc.device)
    mover_of.scatter_(2, torch.where(mover, mover.long().cumsum(2) - 1, torch.full_like(slot, L)), slot)
    src = torch.where(hole, mover_of.gather(2, (hole.long().cumsum(2) - 1).clamp(min=0)), slot)
    width = (keep + ps - 1) // ps
    src = src[..., :width * ps].contiguous()
    valid = (slot < m)[..., :width * ps]
    dest = state["table"].long()[:, :width]
    _plain_evict_one(state["k_pages"], state["k_scale"], state, src, valid, dest, width)
    _plain_evict_one(state["v_pages"], state["v_scale"], state, src, valid, dest, width)
    acc[..., :width * ps] = acc.gather(2, src)
    pos[..., :width * ps] = pos.gather(2, src)
    state["new_lens"].copy_(lens.clamp(max=keep))


# ---------------------------------------------------------------- one pass
def _outputs(state):
    op = state["case"]["op"]
    out = {}
    if op in ("attend", "step"):
        out.update(o=state["o"], lse=state["lse"])
    if op in ("append", "evict"):
        out.update(k_pages=state["k_pages"], v_pages=state["v_pages"], k_scale=state["k_scale"],
                   v_scale=state["v_scale"], new_lens=state["new_lens"])
    if "acc" in state:
        out["acc"] = state["acc"]
    if op == "evict":
        out["positions"] = state["positions"]
    return out


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import exact_io_aware_forward_gb300 as fa
        if "cache" not in state:  # what a serving loop keeps: the cache's handle and the workspace
            state["cache"] = fa.PagedCache(state["k_pages"], state["v_pages"], state["k_scale"], state["v_scale"],
                                           state["table"])
            n = (fa.fa_paged_evict_workspace_size(state["cache"], case["keep"]) if op == "evict" else
                 fa.fa_paged_workspace_size(state["cache"], case["Hq"], case["Nq"], weights=case["weights"]))
            state["workspace"] = torch.empty(max(n, 1), dtype=torch.uint8, device=state["table"].device)
        cache = state["cache"]
        if op in ("append", "step"):
            fa.fa_paged_append(cache, state["k"], state["v"], state["lens"], state["new_lens"], state["counts"],
                               weight_acc=state.get("acc"))
        if op in ("attend", "step"):
            fa.fa_forward_paged(cache, state["q"], state["new_lens"] if op == "step" else state["lens"], state["o"],
                                state["lse"], state["workspace"], causal=True, weight_acc=state.get("acc"))
        if op == "evict":
            # the weights and positions as the steps since the last eviction have left them
            state["acc"].copy_(state["acc_now"])
            state["positions"].copy_(state["positions_now"])
            fa.fa_paged_evict(cache, state["lens"], state["new_lens"], state["acc"], state["positions"],
                              state["workspace"], case["keep"], case["recent"])
    else:
        if op in ("append", "step"):
            _plain_append(state)
        if op in ("attend", "step"):
            _plain_attend(state, state["new_lens"] if op == "step" else state["lens"])
        if op == "evict":
            _plain_evict(state)
    return _outputs(state)


def work(case):
    """Codes, scales, queries and results, each read or written once; two products of the query rows with all slots."""
    B, hkv, hq, nq, d, ps = (case[k] for k in ("B", "Hkv", "Hq", "Nq", "d", "ps"))
    lens, counts = _lens(case), _counts(case)
    slots = sum(lens) + (sum(counts) if case["op"] == "step" else 0)
    pages = sum((n + ps - 1) // ps for n in lens)
    nbytes = flops = 0.0
    if case["op"] in ("attend", "step"):
        nbytes += 2.0 * slots * hkv * d + 8.0 * pages * hkv + 4.0 * pages + B * hq * nq * (4.0 * d + 4)
        nbytes += 8.0 * slots * hkv if case["weights"] else 0
        flops += 4.0 * slots * hq * nq * d
    if case["op"] in ("append", "step"):
        nbytes += sum(counts) * hkv * d * 2.0 * (2 + 1) + 8.0 * hkv * sum(n // ps + 1 for n in counts) + 12.0 * B
        flops += sum(counts) * hkv * d * 4.0
    if case["op"] == "evict":
        for n in lens:
            m, r = min(n, case["keep"]), min(n, (case["recent"] + 1) // 2)  # positions are two apart on average
            behind = max(n - m, 0)  # slots behind the new length: the protected ones and their share of the others move
            moved = 0.0
            if behind:
                moved = min(r, behind) + max(behind - r, 0) * (m - r) / max(n - r, 1)
            nbytes += hkv * (8.0 * n + moved * (4.0 * d + 16))
            flops += hkv * (2.0 * n + 4.0 * d * moved)
    return {"bytes": nbytes, "flops": max(flops, 1.0)}


# ---------------------------------------------------------------- 64 bits
def _exact_sequence(pages, scale, table, b, n, ps):
    """Slots 0 .. n-1 of sequence b in float64, [Hkv, n, d]."""
    idx = table[b, :(n + ps - 1) // ps].long()
    x = pages.view(torch.uint8)[idx].view(pages.dtype).float().double() * scale[idx].double()[:, :, None, None]
    return torch.cat(list(x), 1)[:, :n] if len(idx) else x.new_zeros(pages.shape[1], 0, pages.shape[3])


def _exact_round(x, dtype):
    """To the nearest code, ties to even (values are within the type's range)."""
    return x.float().to(dtype).view(torch.uint8)


def _exact_append(s, case):
    """Page by page: old slots and new ones meet at one scale."""
    ps, kind = case["ps"], case["cache"]
    powers = torch.tensor([2.0 ** e for e in range(-100, 128)], dtype=torch.float64, device=s["k"].device)
    limits = powers * FP8_MAX[kind]
    for b, (n, cnt) in enumerate(zip(_lens(case), _counts(case))):
        for t in range(n // ps, (n + cnt - 1) // ps + 1) if cnt else ():
            p = int(s["table_host"][b][t])
            lo, hi = max(n, t * ps), min(n + cnt, t * ps + ps)
            for pages, scale, x in ((s["k_pages"], s["k_scale"], s["k"]), (s["v_pages"], s["v_scale"], s["v"])):
                val = x[b, :, lo - n:hi - n].double()  # [Hkv, tokens, d]
                amax = val.abs().amax((1, 2))
                # the smallest power 2^e, e >= -100, with amax <= 7/8 * 2^top * 2^e
                new = powers[torch.searchsorted(limits, amax)]
                if n > t * ps:
                    was = scale[p].double()
                    new = torch.maximum(was, new)
                    old = pages[p, :, :n - t * ps].float().double() * (was / new)[:, None, None]
                    pages.view(torch.uint8)[p, :, :n - t * ps] = _exact_round(old, pages.dtype)
                pages.view(torch.uint8)[p, :, lo - t * ps:hi - t * ps] = _exact_round(val / new[:, None, None],
                                                                                    pages.dtype)
                scale[p] = new.float()
        if "acc" in s:
            s["acc"][b, :, n:n + cnt] = 0


def _exact_evict(s, case):
    """Head by head, from the sorted list of its slots."""
    hkv, ps, keep, recent = (case[k] for k in ("Hkv", "ps", "keep", "recent"))
    for b, n in enumerate(_lens(case)):
        m = min(n, keep)
        if n == m:
            continue
        pages = torch.tensor(s["table_host"][b], device=s["acc"].device)
        used = pages[:(m + ps - 1) // ps]
        k_scale, v_scale = s["k_scale"].double(), s["v_scale"].double()
        for h in range(hkv):
            acc, pos = s["acc"][b, h, :n].double(), s["positions"][b, h, :n].long()
            acc[pos > pos.max() - recent] = math.inf
            stays = torch.sort(torch.argsort(-acc, stable=True)[:m])[0]
            src = torch.arange(m, device=acc.device)
            gone = torch.ones_like(src, dtype=torch.bool)
            gone[stays[stays < m]] = False
            src[gone] = stays[stays >= m]
            for x, scale, all_scales in ((s["k_pages"], s["k_scale"], k_scale), (s["v_pages"], s["v_scale"], v_scale)):
                of = all_scales[pages[src // ps], h]
                new = torch.zeros(len(used), dtype=torch.float64, device=acc.device)
                new.index_reduce_(0, torch.arange(m, device=acc.device) // ps, of, "amax")
                code = x.view(torch.uint8)[pages[src // ps], h, src % ps].view(x.dtype).float().double()
                at = torch.arange(m, device=acc.device)
                x.view(torch.uint8)[used[at // ps], h, at % ps] = _exact_round(
                    code * (of / new[at // ps])[:, None], x.dtype)
                scale[used, h] = new.float()
            s["acc"][b, h, :m] = s["acc"][b, h, src]
            s["positions"][b, h, :m] = s["positions"][b, h, src]
    return dict(k_pages=s["k_pages"], v_pages=s["v_pages"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                acc=s["acc"], new_lens=None, positions=None)


def _exact_attend(s, case, lens):
    B, hkv, hq, nq, d, ps = (case[k] for k in ("B", "Hkv", "Hq", "Nq", "d", "ps"))
    g = hq // hkv
    o = torch.zeros(B, hq, nq, d, dtype=torch.float64, device=s["q"].device)
    lse = torch.full((B, hq, nq), -math.inf, dtype=torch.float64, device=o.device)
    acc = s["acc"].double() if "acc" in s else None
    for b, n in enumerate(lens):
        if n == 0:
            continue
        k = _exact_sequence(s["k_pages"], s["k_scale"], s["table"], b, n, ps)
        v = _exact_sequence(s["v_pages"], s["v_scale"], s["table"], b, n, ps)
        for i in range(nq):
            end = n - nq + i + 1  # slots that query i sees
            if end <= 0:
                continue
            qi = s["q"][b, :, i].double().view(hkv, g, d)
            x = torch.einsum("hgd,hnd->hgn", qi, k[:, :end]) / math.sqrt(d)
            z = torch.logsumexp(x, 2)
            w = torch.exp(x - z[..., None])
            o[b, :, i] = torch.einsum("hgn,hnd->hgd", w, v[:, :end]).reshape(hq, d)
            lse[b, :, i] = z.reshape(hq)
            if acc is not None:
                acc[b, :, :end] += w.sum(1)
    return o, lse, acc


def exact(case, seed):
    s = prepare(case, seed)
    s["table_host"] = s["table"].tolist()
    op = case["op"]
    if op == "evict":
        return _exact_evict(s, case)
    if op == "append" and sum(_counts(case)) // case["ps"] + case["B"] > 4000:
        return None
    if op in ("append", "step"):
        _exact_append(s, case)
    lens = [n + c for n, c in zip(_lens(case), _counts(case))] if op != "attend" else _lens(case)
    out = {}
    if op in ("attend", "step"):
        o, lse, acc = _exact_attend(s, case, lens)
        out.update(o=o, lse=lse)
        if acc is not None:
            out["acc"] = acc
    if op == "append":
        out.update(k_pages=s["k_pages"], v_pages=s["v_pages"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                   new_lens=None)
    return out
