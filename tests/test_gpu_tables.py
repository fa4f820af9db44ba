"""Block tables and slot maps from request lengths, and released pages, against a plain sequential form: whole numbers,
equal throughout."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
PAGE = 16


def plain_release(bt, seq, gone, stack, count):
    stack, count = stack.copy(), int(count)
    out = seq.copy()
    for r in range(len(seq)):
        if gone[r]:
            for j in range(-(-int(seq[r]) // PAGE)):
                if count < len(stack):
                    stack[count] = bt[r, j]
                    count += 1
            out[r] = 0
    return stack, count, out


def plain_extend(bt, seq, new, stack, count, slots, pos):
    bt, slots, pos = bt.copy(), slots.copy(), pos.copy()
    R, mp = bt.shape
    off, seq_out, granted = np.zeros(R + 1, np.int64), seq.copy(), np.zeros(R, np.int32)
    taken = wanted = at = 0
    for r in range(R):
        n0, n = int(seq[r]), int(new[r])
        old, need = -(-n0 // PAGE), -(-(n0 + n) // PAGE) - -(-n0 // PAGE)
        fits = old + need <= mp
        need = need if fits else 0
        ok = fits and (need == 0 or wanted + need <= count)
        if ok:
            for k in range(need):
                bt[r, old + k] = stack[count - 1 - wanted - k]
            seq_out[r] = n0 + n
            taken = max(taken, wanted + need) if need else taken
        granted[r] = ok
        wanted += need
        off[r] = at
        for i in range(n):
            if at < len(slots):
                p = n0 + i
                page = bt[r, p // PAGE] if ok else -1
                slots[at] = page * PAGE + p % PAGE if page >= 0 else -1
                pos[at] = p
            at += 1
    off[R] = at
    return bt, off, slots, pos, seq_out, granted, count - taken


def _state(R, mp, lens, free, seed, extra=0):
    rng = np.random.default_rng(seed)
    ids = rng.permutation(R * mp + free).astype(np.int32)
    bt = ids[:R * mp].reshape(R, mp).copy()
    stack = np.full(free + extra, -1, np.int32)
    stack[:free] = ids[R * mp:]
    seq = np.asarray(lens, np.int32)
    return bt, seq, stack


def _run_extend(kap, bt, seq, new, stack, count, cap):
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to("cuda")  # noqa: E731
    R = len(seq)
    i32 = dict(dtype=torch.int32, device="cuda")
    t = dict(block_table=d(bt), seq_len=d(seq), new_tokens=d(np.asarray(new, np.int32)), free_pages=d(stack),
             free_count=torch.tensor([count], **i32), free_count_out=torch.full((1,), -9, **i32),
             tok_offsets=torch.full((R + 1,), -9, **i32),
             slot_out=torch.full((cap,), -9, dtype=torch.int64, device="cuda"), pos_out=torch.full((cap,), -9, **i32),
             seq_len_out=torch.full((R,), -9, **i32), granted=torch.full((R,), -9, **i32))
    kap.kap_extend_tables(**t)
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in t.items()}


CASES = [
    # R, max_pages, lengths, new tokens, free pages, room for tokens beyond the sum
    (1, 1, [0], [1], 1, 0),
    (1, 4, [0], [0], 0, 0),
    (3, 4, [15, 16, 17], [1, 1, 1], 2, 3),
    (4, 8, [0, 31, 32, 33], [40, 1, 0, 31], 20, 0),
    (5, 8, [0, 0, 0, 16, 5], [48, 48, 48, 0, 3], 6, 2),          # the third finds 0 of 3 pages left, the last needs none
    (4, 2, [0, 0, 30, 0], [16, 33, 2, 16], 9, 0),                # the second wants a row longer than the table
    (40, 30, "random", "random", 700, 5),
    (700, 20, "random", "random", 3000, 0),
    (2047, 6, "random", "random", 4000, 1),
    (2049, 6, "random", "random", 1500, 0),                      # two tiles, the pages run out in the first
    (5000, 4, "random", "random", 9000, 7),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"R{c[0]}-mp{c[1]}-free{c[4]}")
def test_extend(kap, case):
    R, mp, lens, new, free, room = case
    rng = np.random.default_rng(R)
    over = lens != "random" and any(-(-(a + b) // PAGE) > mp for a, b in zip(lens, new))
    if lens == "random":
        lens = rng.integers(0, mp * PAGE, R)
        new = np.minimum(rng.integers(0, 40, R) * (rng.random(R) < 0.8), mp * PAGE - lens)
    bt, seq, stack = _state(R, mp, lens, free, R + 1, extra=3)
    cap = int(np.sum(new)) + room
    got = _run_extend(kap, bt, seq, new, stack, free, cap)
    assert kap.kap_device_error() == (2 if over else 0)
    ref = plain_extend(bt, seq, np.asarray(new), stack, free, np.full(cap, -9, np.int64), np.full(cap, -9, np.int32))
    for name, want in zip(("block_table", "tok_offsets", "slot_out", "pos_out", "seq_len_out", "granted"), ref):
        assert np.array_equal(got[name], want), name
    assert int(got["free_count_out"][0]) == ref[6]
    assert np.array_equal(got["free_pages"], stack)


def test_one_long_prompt_among_single_tokens(kap):
    R, mp = 300, 5000
    lens = [7 * r % 100 for r in range(R)]
    new = [1] * R
    new[150] = 70001
    bt, seq, stack = _state(R, mp, lens, 6000, 1)
    cap = sum(new)
    got = _run_extend(kap, bt, seq, new, stack, 6000, cap)
    assert kap.kap_device_error() == 0
    ref = plain_extend(bt, seq, np.asarray(new), stack, 6000, np.full(cap, -9, np.int64), np.full(cap, -9, np.int32))
    for name, want in zip(("block_table", "tok_offsets", "slot_out", "pos_out", "seq_len_out", "granted"), ref):
        assert np.array_equal(got[name], want), name


def test_too_little_room_and_bad_numbers(kap):
    bt, seq, stack = _state(3, 4, [5, 0, 20], 5, 2)
    got = _run_extend(kap, bt, seq, [10, 10, 10], stack, 5, 12)   # 30 tokens, room for 12
    assert kap.kap_device_error() == 2
    ref = plain_extend(bt, seq, np.array([10, 10, 10]), stack, 5, np.full(12, -9, np.int64), np.full(12, -9, np.int32))
    assert np.array_equal(got["slot_out"], ref[2]) and int(got["tok_offsets"][3]) == 30
    # negative lengths count as 0, a count past the stack's capacity as the capacity
    got = _run_extend(kap, bt, np.array([-4, 0, 20], np.int32), [3, -5, 0], stack, 50, 3)
    assert kap.kap_device_error() == 4 | 2
    assert got["tok_offsets"].tolist() == [0, 3, 3, 3] and got["seq_len_out"].tolist() == [3, 0, 20]
    assert int(got["free_count_out"][0]) == 4 and got["block_table"][0, 0] == stack[4]
    # a negative id on the stack: its tokens have no slot
    stack[4] = -3
    got = _run_extend(kap, bt, np.array([0, 0, 20], np.int32), [2, 0, 0], stack, 5, 2)
    assert kap.kap_device_error() == 1
    assert got["slot_out"].tolist() == [-1, -1]


@pytest.mark.parametrize("R,mp", [(1, 1), (33, 9), (2048, 5), (4100, 3)])
def test_release_then_extend(kap, R, mp):
    """A step as a scheduler makes it: finished requests go, their slots take new ones, the others go on."""
    rng = np.random.default_rng(R)
    lens = rng.integers(0, mp * PAGE + 1, R)
    gone = (rng.random(R) < 0.3).astype(np.int32) * 5
    bt, seq, stack = _state(R, mp, lens, 10, 3, extra=R * mp)
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to("cuda")  # noqa: E731
    i32 = dict(dtype=torch.int32, device="cuda")
    st, c1, s1 = d(stack), torch.zeros(1, **i32), torch.zeros(R, **i32)
    kap.kap_release_tables(d(bt), d(seq), d(gone), st, torch.tensor([10], **i32), c1, s1)
    assert kap.kap_device_error() == 0
    stack1, count1, seq1 = plain_release(bt, seq, gone, stack, 10)
    assert np.array_equal(st.cpu().numpy(), stack1) and int(c1) == count1 and np.array_equal(s1.cpu().numpy(), seq1)
    new = np.where(gone > 0, rng.integers(0, mp * PAGE + 1, R), np.minimum(1, mp * PAGE - seq1))
    got = _run_extend(kap, bt, seq1, new, stack1, count1, int(new.sum()))
    ref = plain_extend(bt, seq1, new, stack1, count1, np.full(int(new.sum()), -9, np.int64),
                       np.full(int(new.sum()), -9, np.int32))
    for name, want in zip(("block_table", "tok_offsets", "slot_out", "pos_out", "seq_len_out", "granted"), ref):
        assert np.array_equal(got[name], want), name
    # no page is held twice
    held = [got["block_table"][r, j] for r in range(R) for j in range(-(-int(got["seq_len_out"][r]) // PAGE))]
    left = got["free_pages"][:int(got["free_count_out"][0])].tolist()
    assert len(set(held)) == len(held) and not set(held) & set(left)


def test_release_past_the_capacity(kap):
    bt, seq, stack = _state(2, 4, [64, 33], 3, 2, extra=4)
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to("cuda")  # noqa: E731
    i32 = dict(dtype=torch.int32, device="cuda")
    st, c1, s1 = d(stack), torch.zeros(1, **i32), torch.zeros(2, **i32)
    kap.kap_release_tables(d(bt), d(seq), torch.ones(2, **i32), st, torch.tensor([3], **i32), c1, s1)
    assert kap.kap_device_error() == 2
    ref = plain_release(bt, seq, [1, 1], stack, 3)
    assert np.array_equal(st.cpu().numpy(), ref[0]) and int(c1) == 7 and s1.cpu().tolist() == [0, 0]


def test_binding_refusals(kap):
    i32 = dict(dtype=torch.int32, device="cuda")
    a = dict(block_table=torch.zeros(2, 3, **i32), seq_len=torch.zeros(2, **i32), new_tokens=torch.zeros(2, **i32),
             free_pages=torch.zeros(4, **i32), free_count=torch.zeros(1, **i32), free_count_out=torch.zeros(1, **i32),
             tok_offsets=torch.zeros(3, **i32), slot_out=torch.zeros(5, dtype=torch.int64, device="cuda"),
             pos_out=torch.zeros(5, **i32), seq_len_out=torch.zeros(2, **i32), granted=torch.zeros(2, **i32))
    kap.kap_extend_tables(**a)
    for bad in (dict(slot_out=a["pos_out"]), dict(seq_len=a["seq_len"].long())):
        with pytest.raises(TypeError):
            kap.kap_extend_tables(**{**a, **bad})
    for bad in (dict(tok_offsets=torch.zeros(2, **i32)), dict(pos_out=torch.zeros(4, **i32)),
                dict(block_table=torch.zeros(6, **i32)), dict(granted=torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            kap.kap_extend_tables(**{**a, **bad})
    for bad in (dict(seq_len_out=a["seq_len"]), dict(free_count_out=a["free_count"])):   # aliased
        with pytest.raises(kap.KapError) as e:
            kap.kap_extend_tables(**{**a, **bad})
        assert e.value.status == -1
    with pytest.raises(kap.KapError) as e:
        kap.kap_release_tables(a["block_table"], a["seq_len"], a["granted"], a["free_pages"], a["free_count"],
                               a["free_count_out"], a["seq_len"])
    assert e.value.status == -1
