"""The packed kernel's mbarrier protocol (csrc/group_tc.cu) on the CPU, with the randomized
model of barrier_model.py: its ring of unit parts, its query tiles that scan different
numbers of key tiles, and V rows that softmax warps zero in shared memory before both
tiles' value contractions read them.

Besides what that model tracks in tensor memory, shared memory is named here: ("K", slot)
and ("V", slot) hold the key tile that the loading warp put there, ("Z", slot, w) the tile
whose rows behind the entry's end warp w of a softmax group has zeroed, ("Q", t) the part
whose queries it is, ("part", slot) the part that the ring's slot describes.  A load counts
as overwriting its slot when it is issued.

A part is (n, need): key tiles that each query tile scans (0: none), and whether the last
of them has V rows to zero (for a tile that scans the part's last key tile)."""
import random

import pytest

from barrier_model import Barrier, TensorCore, run

T = (0, 1)
W = range(4)


def zeroing_tile(n, need):
    """The query tile that zeroes rows of the part's last V tile: the one whose value
    contraction comes first among those that need it; None: nobody."""
    last = max(n) - 1
    for t in T:
        if need[t] and n[t] - 1 == last:
            return t
    return None


def protocol(parts, rng, kstages=2, vstages=3, ring=4, part_readers=9, zero_by=None):
    tc = TensorCore()
    bar = lambda name, count=1: Barrier(name, count)  # noqa: E731
    q_full, q_empty, s_full, o_done = ([bar(f"{x}[{t}]") for t in T] for x in ("q_full", "q_empty", "s_full", "o_done"))
    p_full, o_free = ([bar(f"{x}[{t}]", 4) for t in T] for x in ("p_full", "o_free"))
    k_full, k_empty = ([bar(f"{x}[{s}]") for s in range(kstages)] for x in ("k_full", "k_empty"))
    v_empty = [bar(f"v_empty[{s}]") for s in range(vstages)]
    seg_full = [bar(f"seg_full[{s}]") for s in range(ring)]
    seg_empty = [bar(f"seg_empty[{s}]", part_readers) for s in range(ring)]

    def producer():
        uses, kn = [0, 0], 0
        for i, part in enumerate(parts + [None]):
            s = i % ring
            yield ("wait", seg_empty[s], ((i // ring) & 1) ^ 1)
            yield ("write", ("part", s), i)
            yield ("arrive", seg_full[s], i)
            if part is None:
                return
            n, _ = part
            for t in T:
                if n[t]:
                    yield ("wait", q_empty[t], (uses[t] & 1) ^ 1)
                    uses[t] += 1
                    yield ("write", ("Q", t), i)
                    yield ("arrive_tx", q_full[t], i, 1)
            for j in range(max(n)):
                yield ("wait", k_empty[kn % kstages], ((kn // kstages) & 1) ^ 1)
                yield ("wait", v_empty[kn % vstages], ((kn // vstages) & 1) ^ 1)
                yield ("write", ("K", kn % kstages), (i, j))
                yield ("write", ("V", kn % vstages), (i, j))
                yield ("arrive_tx", k_full[kn % kstages], kn, 2)
                kn += 1

    def issuer():
        qc, pc, of, kn, vn = [0, 0], [0, 0], [1, 1], 0, 0
        for i, part in enumerate(parts + [None]):
            s = i % ring
            yield ("wait", seg_full[s], (i // ring) & 1)
            yield ("read", ("part", s), i)
            yield ("arrive", seg_empty[s], i)
            if part is None:
                return
            n, need = part
            zero = zeroing_tile(n, need)

            def score(t, j, k):
                yield ("mma", [(("Q", t), i), (("K", k % kstages), (i, j))], [(("S", t, w), ("S", i, j)) for w in W])
                yield ("commit", s_full[t], (i, j))

            for t in T:
                if n[t]:
                    yield ("wait", q_full[t], qc[t])
                    qc[t] ^= 1
                    yield ("wait", k_full[kn % kstages], (kn // kstages) & 1)
                    yield from score(t, 0, kn)
                    if n[t] == 1:
                        yield ("commit", q_empty[t], i)
            kn += 1
            yield ("commit", k_empty[(kn - 1) % kstages], kn - 1)
            for j in range(max(n)):
                vs, nxt, have = vn % vstages, kn, False
                vn += 1
                for t in T:
                    if j >= n[t]:
                        continue
                    yield ("wait", p_full[t], pc[t])
                    pc[t] ^= 1
                    if j == 0:
                        yield ("wait", o_free[t], of[t])
                        of[t] ^= 1
                    reads = [(("S", t, w), ("P", i, j)) for w in W] + [(("V", vs), (i, j))]
                    if j:
                        reads += [(("U", t, w), ("U", i, j - 1)) for w in W]
                    if need[t] and j == n[t] - 1 == max(n) - 1 and zero is not None:
                        reads += [(("Z", vs, w), (i, j)) for w in W]
                    yield ("mma", reads, [(("U", t, w), ("U", i, j)) for w in W])
                    if j == n[t] - 1:
                        yield ("commit", o_done[t], i)
                    if j + 1 < n[t]:
                        if not have:
                            yield ("wait", k_full[nxt % kstages], (nxt // kstages) & 1)
                            have = True
                        yield from score(t, j + 1, nxt)
                        if j + 1 == n[t] - 1:
                            yield ("commit", q_empty[t], i)
                yield ("commit", v_empty[vs], vn - 1)
                if have:
                    kn += 1
                    yield ("commit", k_empty[nxt % kstages], nxt)

    def softmax(t, w):
        sc = oc = base = 0
        for i, part in enumerate(parts + [None]):
            s = i % ring
            yield ("wait", seg_full[s], (i // ring) & 1)
            yield ("read", ("part", s), i)
            if part is None:
                return
            n, need = part
            first, base = base, base + max(n)
            zero = zeroing_tile(n, need) if zero_by is None else zero_by
            if n[t] == 0:
                yield ("work",)
                yield ("read", ("part", s), i)
                yield ("arrive", seg_empty[s], i)
                continue
            for j in range(n[t]):
                yield ("read", ("part", s), i)
                yield ("wait", s_full[t], sc)
                sc ^= 1
                yield ("read", ("S", t, w), ("S", i, j))
                if need[t] and j == max(n) - 1 and t == zero:
                    vs = (first + j) % vstages
                    yield ("read", ("V", vs), (i, j))
                    yield ("write", ("Z", vs, w), (i, j))
                if j and rng.random() < 0.3:  # a rescale
                    yield ("read", ("U", t, w), ("U", i, j - 1))
                    yield ("write", ("U", t, w), ("U", i, j - 1))
                for _ in range(rng.randint(1, 5)):
                    yield ("work",)
                yield ("write", ("S", t, w), ("P", i, j))
                yield ("arrive", p_full[t], (i, j))
            yield ("read", ("part", s), i)
            yield ("arrive", seg_empty[s], i)
            yield ("wait", o_done[t], oc)
            oc ^= 1
            for _ in range(rng.randint(1, 4)):
                yield ("read", ("U", t, w), ("U", i, n[t] - 1))
            yield ("arrive", o_free[t], i)

    roles = {"producer": producer(), "issuer": issuer()}
    for t in T:
        roles.update({f"sm{t}.{w}": softmax(t, w) for w in W})
    return roles, tc


def random_parts(rng):
    parts = []
    for _ in range(rng.randint(1, 9)):
        n0 = rng.choice([0, 1, 1, 1, 2, 3, 5])
        n1 = rng.choice([0, n0, n0, n0 + 1, 1, 2])  # a tile without rows, or one key tile more
        if n0 == n1 == 0:
            n0 = 1
        last = max(n0, n1)
        parts.append(((n0, n1), (n0 == last and rng.random() < 0.5, n1 == last and rng.random() < 0.7)))
    return parts


def explore(trials, seed, parts_of=random_parts, **kw):
    rng = random.Random(seed)
    for _ in range(trials):
        parts = parts_of(rng)
        roles, tc = protocol(parts, rng, **kw)
        violations, deadlocked = run(roles, tc, rng)
        if violations or deadlocked:
            return parts, violations, deadlocked
    return None


@pytest.mark.parametrize("kstages,vstages", [(2, 3), (4, 4)])  # D = 128, D = 64
def test_the_protocol(kstages, vstages):
    assert explore(500, 41, kstages=kstages, vstages=vstages) is None


def test_many_short_parts():
    """More parts in flight than the ring holds: single tiles, as packed short prompts have."""
    assert explore(300, 42, lambda r: [((1, r.choice([0, 1])), (False, False)) for _ in range(r.randint(5, 14))]) is None


def test_the_model_finds_a_part_given_back_too_early():
    """Planted: the ring's slot counts one reader less than there are."""
    found = explore(400, 43, part_readers=8)
    assert found is not None


def test_the_model_finds_rows_zeroed_by_the_later_tile():
    """Planted: where both tiles scan the last key tile, the second one zeroes V's rows."""
    both = lambda r: [((n, n), (True, True)) for n in (r.choice([1, 2]) for _ in range(3))]  # noqa: E731
    assert explore(300, 44, both) is None
    found = explore(300, 44, both, zero_by=1)
    assert found is not None and any("('Z', " in v for v in found[1])


def test_the_model_finds_too_few_value_slots():
    """Planted: one V slot.  The next key tile lands as a whole (its K and V on one barrier) and
    its scores are issued before V of this one is given back."""
    found = explore(300, 45, vstages=1)
    assert found is not None and found[2] and not found[1]
    assert explore(300, 45, vstages=2) is None
