"""Plain model of the page operators, one entry at a time in Python integers: what
sra_kv_fork_rows, sra_kv_resize_rows, sra_kv_compact_pages and sra_kv_copy_pages do to the
state and to the caches. State: numpy int64 arrays ``table`` [rows, M], ``seq`` [rows] and ``ref``
[num_blocks]; caches: a list of torch CPU tensors [2, num_blocks, bs, n_kv, hd], moved as bits.
Every function returns the count of errors."""
import numpy as np


def pages(L, bs):
    return -(-int(L) // bs)


def bits(c):
    """The cache as integers (NaN patterns are moved as they are)."""
    return c.view({2: __import__("torch").int16, 4: __import__("torch").int32}[c.element_size()])


class State:
    def __init__(self, table, seq, ref, bs):
        self.table = np.array(table, dtype=np.int64)
        self.seq, self.ref, self.bs = np.array(seq, dtype=np.int64), np.array(ref, dtype=np.int64), bs

    @property
    def cap(self):
        return self.table.shape[1] * self.bs

    def drop(self, page):
        """One holder less; a page out of range or without holders is an error."""
        if not 0 <= page < len(self.ref) or self.ref[page] <= 0:
            return 1
        self.ref[page] -= 1
        return 0

    def consistent(self):
        """Whether the counts are the rows' used entries."""
        want = np.zeros_like(self.ref)
        for row, L in zip(self.table, self.seq):
            for p in row[:pages(L, self.bs)]:
                want[p] += 1
        return bool((want == self.ref).all())


def copy(caches, src, dst):
    errors = 0
    before = [bits(c).clone() for c in caches]
    for s, d in zip(src, dst):
        if s < 0 or d < 0:
            continue
        if s >= caches[0].shape[1] or d >= caches[0].shape[1]:
            errors += int(s != d)
            continue
        for c, b in zip(caches, before):
            bits(c)[:, d] = b[:, s]
    return errors


def fork(st, parents, children):
    errors = 0
    R, bs = len(st.seq), st.bs
    table, seq = st.table.copy(), st.seq.copy()
    todo = []
    for i, (p, c) in enumerate(zip(parents, children)):
        if p < 0 or c < 0:
            continue
        if p >= R or c >= R or c in list(children[:i]) or not 0 <= seq[p] <= st.cap or not 0 <= seq[c] <= st.cap:
            errors += 1
            continue
        todo.append((p, c))
        for e in table[p, :pages(seq[p], bs)]:
            if 0 <= e < len(st.ref):
                st.ref[e] += 1
            else:
                errors += 1
    for p, c in todo:
        for e in table[c, :pages(seq[c], bs)]:
            errors += st.drop(e)
        k = pages(seq[p], bs)
        st.table[c] = -1
        st.table[c, :k] = table[p, :k]
        st.seq[c] = seq[p]
    return errors


def resize(st, rows, lens, caches):
    """Returns (errors, pos, slot)."""
    errors = 0
    bs, R, NB = st.bs, len(st.seq), len(st.ref)
    act = []
    for i, (r, L) in enumerate(zip(rows, lens)):
        if r < 0:
            continue
        if r >= R or r in list(rows[:i]) or not 0 <= L <= st.cap or not 0 <= st.seq[r] <= st.cap:
            errors += 1
            continue
        act.append((i, r, int(L), int(st.seq[r])))
    for i, r, L, old in act:
        for j in range(pages(L, bs), pages(old, bs)):
            errors += st.drop(st.table[r, j])
            st.table[r, j] = -1
    plan, upto = [], 0
    ok = {}
    for i, r, L, old in act:
        ok[i] = True
        if L <= old:
            st.seq[r] = L
            continue
        need, src = pages(L, bs) - pages(old, bs), -1
        if old % bs:
            last = int(st.table[r, pages(old, bs) - 1])
            if not 0 <= last < NB:
                errors += 1
                ok[i] = False
                continue
            if st.ref[last] > 1:
                src, need = last, need + 1
        upto += need
        plan.append((i, r, L, old, src, need, upto))
    free = [p for p in range(NB) if st.ref[p] <= 0]
    for i, r, L, old, src, need, upto in plan:
        if need and upto > len(free):
            errors += 1
            continue
        given = free[upto - need:upto]
        begin = pages(old, bs)
        if src >= 0:
            begin -= 1
            st.ref[src] -= 1
            for c in caches:
                bits(c)[:, given[0], :old % bs] = bits(c)[:, src, :old % bs]
        for j, p in enumerate(given):
            st.table[r, begin + j] = p
            st.ref[p] = 1
        st.seq[r] = L
    pos, slot = np.full(len(rows), -1), np.full(len(rows), -1)
    for i, r, *_ in act:
        L = int(st.seq[r])
        if ok[i] and L > 0:
            page = int(st.table[r, (L - 1) // bs])
            pos[i] = L - 1
            slot[i] = page * bs + (L - 1) % bs if 0 <= page < NB else -1
    return errors, pos, slot


def compact(st, caches):
    """Returns (errors, live pages)."""
    errors = 0
    live = [p for p in range(len(st.ref)) if st.ref[p] > 0]
    n = len(live)
    src = [p for p in live if p >= n]
    dst = [p for p in range(n) if st.ref[p] <= 0]
    to = dict(zip(src, dst))
    alive = set(live)
    for row, L in zip(st.table, st.seq):
        if not 0 <= L <= st.cap:
            errors += 1
            continue
        for j in range(pages(L, st.bs)):
            if int(row[j]) not in alive:
                errors += 1
            else:
                row[j] = to.get(int(row[j]), row[j])
    for s, d in to.items():
        st.ref[d], st.ref[s] = st.ref[s], 0
        for c in caches:
            bits(c)[:, d] = bits(c)[:, s]
    return errors, n
