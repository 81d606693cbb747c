"""The waits of the attention over 8-bit pages (paged_attn_q8.cu) on the CPU: a
model of its roles and barriers under random schedules.

A barrier counts arrivals and flips its phase when all of one phase are there;
a wait for a parity passes when the current phase has the other one. The model
has the walk, the two teams of converting warps, the two streams' products and
softmax, and products that end in the order of their issue, some time later. What it
checks is that nothing is written while it is still to be read: a place of the ring
of fp16 halves, and the second stream's queries, which lie over the last raw places.
"""
import ctypes
import os
import random
import re
import shutil
import subprocess

import pytest

from block_diffusion_drafter_pass_gb300 import _build


@pytest.fixture(scope="module")
def rings(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("rings")
    src, lib = os.path.join(d, "rings.cpp"), os.path.join(d, "rings.so")
    with open(src, "w") as f:
        f.write('#include "paged_q8_rings.h"\nextern "C" {\n'
                "int read_bar(int h, int s) { return dfl::read_bar(h, s); }\n"
                "int free_bar(int h, int s) { return dfl::free_bar(h, s); }\n"
                "int free_parity(int h, int s) { return dfl::free_parity(h, s); }\n}\n")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", _build.CSRC, src, "-o", lib], check=True)
    return ctypes.CDLL(lib)


class Bar:
    def __init__(self, count):
        self.count = self.left = count
        self.phase = 0

    def arrive(self):
        self.left -= 1
        assert self.left >= 0, "more arrivals than a phase has"
        if self.left == 0:
            self.phase += 1
            self.left = self.count

    def passed(self, parity):
        return (self.phase & 1) != parity


class Written(AssertionError):
    pass


def halves(nj, pair):
    """An item's halves in the order that all roles follow: (is keys, step)."""
    lead = 1 if pair else 2
    for i in range(1 - 2 * lead, 2 * nj):
        keys = i & 1
        j = (i >> 1) + (lead if keys else 0)
        if 0 <= j < nj:
            yield bool(keys), j


class Model:
    """One CTA's run over `items` (steps, pair). slots, raw, raw_pair as in the
    kernel's Cfg; `asks_note`: the walk also waits for the pair's queries to be in."""

    def __init__(self, rng, items, slots, raw, raw_pair, release, asks_note=True):
        self.rng, self.items, self.S, self.raw, self.raw_pair = rng, items, slots, raw, raw_pair
        self.asks_note = asks_note
        self.read_bar, self.free_wait = release
        n_bars = 2 * slots
        self.raw_full, self.raw_empty = [Bar(1) for _ in range(raw)], [Bar(1) for _ in range(raw)]
        self.note_full, self.note_empty = [Bar(1) for _ in range(2)], [Bar(2) for _ in range(2)]   # the teams
        self.meet = Bar(2)
        self.kv_full = [[Bar(1) for _ in range(slots)] for _ in range(2)]
        self.kv_empty = [Bar(2) for _ in range(n_bars)]
        self.q_full, self.q_empty = Bar(2), Bar(2)
        self.s_full, self.p_full, self.turn = [Bar(1), Bar(1)], [Bar(1), Bar(1)], [Bar(1), Bar(1)]
        self.pipe = []                     # products in flight, in order
        self.unread = {}                   # slot -> halves' readers still to come
        self.queries = None                # the pair item whose queries lie over raw places, until its scores are done
        self.scored = {}                   # item -> streams whose scores are done
        self.takes = {k: [[rng.random() < 0.8 for _ in range(nj)] for _ in range(2)] for k, (nj, _) in enumerate(items)}

    # --- roles: generators of what they wait for ---
    def walk(self):
        at, used, places = 0, [0] * self.raw, self.raw
        for k, (nj, pair) in enumerate(self.items):
            was, places = places, self.raw_pair if pair else self.raw
            if places > was:
                if self.asks_note:
                    yield lambda: self.note_empty[(k - 1) & 1].passed((k - 1) >> 1 & 1)
                yield lambda: self.q_empty.passed((k - 1) & 1)
            at = 0 if at >= places else at
            yield lambda: self.note_empty[k & 1].passed((k >> 1 & 1) ^ 1)
            self.note_full[k & 1].arrive()
            for _ in halves(nj, pair):
                yield lambda: self.raw_empty[at].passed(used[at] ^ 1)
                if at >= self.raw_pair and self.queries is not None:
                    raise Written(f"codes of item {k} over the queries of item {self.queries}")
                self.raw_full[at].arrive()
                used[at] ^= 1
                at = at + 1 if at + 1 < places else 0

    def team(self, me):
        at, used, half = 0, [0] * self.raw, 0
        for k, (nj, pair) in enumerate(self.items):
            yield lambda: self.note_full[k & 1].passed(k >> 1 & 1)
            places = self.raw_pair if pair else self.raw
            at = 0 if at >= places else at
            if k > 0:
                yield lambda: self.q_empty.passed((k - 1) & 1)
            self.meet.arrive()
            yield lambda: self.meet.passed(k & 1)
            if pair:
                assert self.queries in (None, k)
                self.queries = k
            yield lambda: True   # while they are written
            self.q_full.arrive()
            self.note_empty[k & 1].arrive()
            for keys, j in halves(nj, pair):
                place, h = at, half
                parity = used[at]
                half += 1
                used[at] ^= 1
                at = at + 1 if at + 1 < places else 0
                if h % 2 != me:
                    continue
                yield lambda: self.raw_full[place].passed(parity)
                wait = self.free_wait(h)
                if wait:
                    yield lambda: self.kv_empty[wait[0]].passed(wait[1])
                slot = h % self.S
                if self.unread.get(slot):
                    raise Written(f"half {h} over {self.unread[slot]}")
                self.unread[slot] = [(h, s) for s in (0, 1) if pair or j % 2 == s]
                yield lambda: True   # while it is written
                self.raw_empty[place].arrive()
                for s in (0, 1):
                    if pair or j % 2 == s:
                        self.kv_full[s][slot].arrive()

    def read(self, h, s):
        self.unread[h % self.S].remove((h, s))
        self.kv_empty[self.read_bar(h)].arrive()

    def issue(self, *done):
        self.pipe.append(done)

    def ends(self):
        """Products end in order, some time after they were issued."""
        while True:
            yield lambda: bool(self.pipe)
            for f, *args in self.pipe.pop(0):
                f(*args)

    def scores_done(self, k, s):
        if self.queries == k:
            self.scored.setdefault(k, set()).add(s)
            if len(self.scored[k]) == 2:
                self.queries = None
        self.q_empty.arrive()

    def products(self, s):
        c, np, turns = 0, 0, 0
        got = [0] * self.S

        def there(slot):
            return self.kv_full[s][slot].passed(got[slot])

        for k, (nj, pair) in enumerate(self.items):
            yield lambda: self.q_full.passed(k & 1)
            if not pair:
                order = list(halves(nj, pair))
                for j in range(s, nj, 2):
                    for keys in (True, False):
                        h = c + order.index((keys, j))
                        slot = h % self.S
                        yield lambda: there(slot)
                        got[slot] ^= 1
                        if not keys:
                            yield lambda: self.p_full[s].passed(np & 1)
                            np += 1
                        done = [(self.read, h, s)] + [(self.kv_empty[self.read_bar(h)].arrive,)]
                        if keys:
                            done.append((self.s_full[s].arrive,))
                            if j + 2 >= nj:
                                done.append((self.scores_done, k, s))
                        self.issue(*done)
                if s >= nj:
                    self.issue((self.scores_done, k, s))
            else:
                for j in range(-1, nj):
                    v, key = j >= 0, j + 1 < nj
                    hv, hk = c, c + (1 if v else 0)
                    vs, ks = hv % self.S, hk % self.S
                    if v:
                        yield lambda: there(vs)
                        yield lambda: self.p_full[s].passed(np & 1)
                    if key:
                        yield lambda: there(ks)
                    if s == 1 or turns > 0:
                        par = (turns if s == 1 else turns - 1) & 1
                        yield lambda: self.turn[s].passed(par)
                    turns += 1
                    if v:
                        got[vs] ^= 1
                        np += 1
                        if self.takes[k][s][j]:
                            self.issue((self.read, hv, s))
                        else:
                            self.read(hv, s)
                        yield lambda: True
                    if key:
                        got[ks] ^= 1
                    self.turn[s ^ 1].arrive()
                    if key:
                        if self.takes[k][s][j + 1]:
                            self.issue((self.read, hk, s), (self.s_full[s].arrive,))
                        else:
                            self.s_full[s].arrive()
                            self.read(hk, s)
                    if j + 2 == nj:
                        self.issue((self.scores_done, k, s))
                    c = hk + (1 if key else 0)
            if not pair:
                c += 2 * nj

    def softmax(self, s):
        ns = 0
        for nj, pair in self.items:
            for j in range(nj):
                if pair or j % 2 == s:
                    yield lambda: self.s_full[s].passed(ns & 1)
                    yield lambda: True
                    self.p_full[s].arrive()
                    ns += 1

    def run(self):
        roles = [self.walk(), self.team(0), self.team(1), self.products(0), self.products(1), self.softmax(0),
                 self.softmax(1), self.ends()]
        slow = [self.rng.choice((1, 1, 3, 10, 30)) for _ in roles]
        waits = [lambda: True] * len(roles)
        live = set(range(len(roles)))
        while live - {7}:
            ready = [i for i in live if waits[i]()]
            assert ready, "all roles wait"
            i = self.rng.choices(ready, [1.0 / slow[i] for i in ready])[0]
            try:
                waits[i] = next(roles[i])
            except StopIteration:
                live.discard(i)
        while self.pipe:
            next(roles[7])


def some_items(rng):
    return [(rng.choice((1, 1, 1, 2, 2, 3, 5, 9)), rng.random() < 0.5) for _ in range(rng.randint(1, 14))]


def one_each(S):
    """One barrier a slot, as it was: the phase by the half's turn in its slot."""
    return (lambda h: h % S), (lambda h: (h % S, (h // S & 1) ^ 1))


def of_header(rings, S):
    return (lambda h: rings.read_bar(h, S)), (lambda h: (rings.free_bar(h, S), rings.free_parity(h, S)) if h >= S else None)


SHAPES = {128: (3, 4, 2), 64: (6, 6, 4)}   # slots, raw places, those of a pair


def faults(make, n=400):
    found = {}
    for seed in range(n):
        rng = random.Random(seed)
        try:
            make(rng, some_items(rng)).run()
        except Written as e:
            what = "queries" if "queries" in str(e) else "ring"
            found[what] = found.get(what, 0) + 1
    return found


@pytest.mark.parametrize("d", [64, 128])
def test_nothing_is_written_before_it_is_read(rings, d):
    assert faults(lambda rng, items: Model(rng, items, *SHAPES[d], of_header(rings, SHAPES[d][0]))) == {}


def test_the_model_finds_waits_that_pass_too_early(rings):
    """What each of the two waits is there for."""
    assert "queries" in faults(lambda rng, items: Model(rng, items, *SHAPES[128], of_header(rings, 3), asks_note=False))
    assert "ring" in faults(lambda rng, items: Model(rng, items, *SHAPES[128], one_each(3)))


def kernel():
    with open(os.path.join(_build.CSRC, "paged_attn_q8.cu")) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_the_shapes_are_the_kernels():
    text = kernel()
    assert re.search(r"kSlots = D == 128 \? 3 : 6;", text) and re.search(r"kRawSlots = D == 128 \? 4 : 6, kRawPair = kRawSlots - 2;", text)


def test_the_walk_asks_for_a_pairs_queries_first():
    """Behind a pair it waits for the pair's queries to be in (whose writers have waited for the
    scores before them), and only then for the pair's own scores, whose parity is that of two items before."""
    m = re.search(r"if \(places > was\) \{(.*?)\n        \}", kernel(), re.S)
    assert m, "the walk's wait behind a pair"
    note, scores = m.group(1).find("note_empty"), m.group(1).find("q_empty")
    assert 0 <= note < scores and re.search(r"\(k - 1\) >> 1 & 1", m.group(1)[:scores])


def test_the_ring_is_waited_for_as_modelled():
    """Every arrival and the one wait for a half that was read go by the header's barriers."""
    text = kernel()
    assert "kv_empty[2 * S]" in text and "s < 2 * S; ++s) mbar_init(&kv_empty[s], 2)" in text
    assert re.search(r"half >= S && !wait\(smem_u32\(kv_empty\) \+ free_bar\(half, S\) \* 8, free_parity\(half, S\)\)", text)
    assert len(re.findall(r"bar_(?:commit|arrive)\(empty_of\(", text)) == 6 and "empty_at + slot" not in text


def test_scales_are_fenced_before_their_place_is_copied_into_again():
    """The scale warp's own accesses to a place lie before a proxy fence, and that before the arrival from
    which, by way of the other roles, the next bulk copy into the place follows."""
    text = kernel()
    role = text[text.index("warp == kScaleWarp) {"):text.index("const int s = warp_uniform(warp - kMmaWarp0);")]
    last = max(role.rindex("st.shared.b32"), role.rindex("load_shared_u32"))
    fence, arrive = role.find("fence_proxy_async_smem()"), role.index("bar_arrive(smem_u32(scale_full)")
    assert last < fence < arrive
