"""Write nt_loop.inc: the K loops of the large tiles of nt_loop.h as GCN assembly
text for gfx950.

The C++ part sets up addresses and runs the epilogue; the loop is written
instruction by instruction, because the compiler neither keeps sums, fragments
and prefetches of a 128 x 64 wavefront tile within 256 registers nor keeps the
products between the reads that they hide.

A loop sums a block tile of 16 MT WM x 16 NT WN over steps of 128 bytes of K.
Two to four stages lie in LDS; a stage is A's panel and B's (rows of 128 bytes,
16-byte chunk c of row r in slot c ^ ((r / 2) % 8)), and behind all stages lie
the scales of each one's rows (4 bytes each).

A step's MT x NT products are taken in four quarters, two halves of A by two of
B, in the order (0, x) (0, y) (1, y) (1, x), with x = 0, y = 1 in every other
step and the reverse in between: each quarter but the first of a step changes
one half only, and what it needs is read during the quarter before it, over the
step's end too.  The step's only barrier is at the end of the third quarter, when
all wavefronts have made their last reads of its stage and the next step's loads
have arrived; behind it the loads into that stage start, as many steps ahead as
there are stages.

The loop is unrolled over the stages and both orders (2, 4 or 6 positions) and
entered where it has to be for the last step to be in the last position.  Loads
of steps that do not exist go through descriptors of zero bytes: they touch no
memory, so all steps are alike.  The last step, where K may end within the 128
bytes, and the one before it have code of their own.

Kinds:
  e8m0   8-bit products, power-of-two scales applied by the instruction
  f32u   8-bit products summed from zero, then added times the product of A's
         row's scale and the one scale of the wavefront's B rows
  f32n   the same with a scale for each of B's rows
  pair   numbers as pairs of halfs (64 bytes hi, 64 bytes lo), three products
  w32u, w32n, w8u, w8n
         8-bit codes widened to halfs, four products, scaled afterwards as f32u
         and f32n; the scales floats (w32) or bytes (w8), which a thread each
         turns into floats on their way to LDS
Products that are scaled afterwards lie in a ring of four results, and each is
added when enough more have been issued for it to have arrived.

Widening takes as many vector instructions as scaling does, so fragments are
widened once a step: a half of A and all of B stay widened, and the codes of one
half of each side are on their way.  Those of a step have all been read after
its second quarter, where the barrier is then.

Run as a script to rewrite nt_loop.inc; a test checks that the committed file
is what this writes.
"""

from __future__ import annotations

import os

OUT = os.path.join(os.path.dirname(os.path.abspath(__file__)), "nt_loop.inc")


class Loop:
    """One loop's text.  Registers: v[0:..] the sums, (j MT + i) 4; then the
    fragments of A and B, the widened ones, the ring of results, A's and B's
    scales."""

    def __init__(self, kind, mt, nt, wm, wn, stages):
        self.kind, self.mt, self.nt, self.wm, self.wn, self.stages = kind, mt, nt, wm, wn, stages
        self.positions = stages if stages % 2 == 0 else 2 * stages
        self.hm, self.hn = mt // 2, nt // 2
        self.waves = wm * wn
        self.bm, self.bn = 16 * mt * wm, 16 * nt * wn
        self.la, self.lb = self.bm // 8 // self.waves, self.bn // 8 // self.waves
        self.stride = 128 * (self.bm + self.bn)  # bytes from one stage to the next
        self.scaled = kind != "pair"
        self.wide = kind[0] == "w"
        self.after = self.wide or kind[0] == "f"
        self.uniform = self.after and kind[-1] == "u"
        self.rows = self.after and kind[-1] == "n"
        self.bytes = kind.startswith("w8")
        # loads of 64 scales a wavefront
        self.scale_loads = -(-((self.bm + self.bn) // 64) // self.waves) if self.scaled else 0
        self.scale_stage = 256 * self.waves * self.scale_loads
        # products after which a result has arrived, and the first of a quarter
        # after which no scales of the quarter before are wanted
        self.age = 5 if self.wide else 3
        self.settled = 6 if self.wide else 2
        at = 4 * mt * nt
        # slots for A: all of MT, or half of it, each used again when its products are issued
        self.slots = mt if mt <= 4 and not self.wide else self.hm
        self.a0, at = at, at + 8 * self.slots
        self.b0, at = at, at + 8 * (self.hn if self.wide else nt)
        self.wa0, at = at, at + (16 * self.hm if self.wide else 0)
        self.wb0, at = at, at + (16 * nt if self.wide else 0)
        self.t0, at = at, at + (16 if self.after else 0)
        self.sm0, at = at, at + (mt if self.scaled else 0)
        self.sn0, at = at, at + (4 * nt if self.rows else 2 if self.uniform else nt if self.scaled else 0)
        self.sv, at = at, at + (stages if self.bytes else 0)
        self.registers = at
        self.lines = []
        self.reads = []    # LDS reads under way, oldest first: what arrives
        self.pending = []  # products not yet added: (result, j, i, issued)
        self.count = 0     # products (of a sum of their own) so far
        self.issued = 0    # matrix instructions so far

    # -- text

    def emit(self, text):
        self.lines.append(text)

    def acc(self, j, i):
        at = 4 * (j * self.mt + i)
        return f"v[{at}:{at + 3}]"

    def fa(self, i, part=None):
        return self._frag(self.a0 + 8 * (i % self.slots), part)

    def fb(self, j, part=None):
        return self._frag(self.b0 + 8 * (j % self.hn if self.wide else j), part)

    def wa(self, i, q):
        at = self.wa0 + 16 * (i % self.hm) + 4 * q
        return f"v[{at}:{at + 3}]"

    def wb(self, j, q):
        at = self.wb0 + 16 * j + 4 * q
        return f"v[{at}:{at + 3}]"

    @staticmethod
    def _frag(at, part):
        if part is None:
            return f"v[{at}:{at + 7}]"
        return f"v[{at + 4 * part}:{at + 4 * part + 3}]"

    def sm(self, i):
        return f"v{self.sm0 + i}"

    def sn(self, j, r=0):
        return f"v{self.sn0 + (4 * j + r if self.rows else j)}"

    # -- LDS reads; `name` says what arrives with them

    def read(self, text, name):
        self.emit(text)
        self.reads.append(name)

    def need(self, names):
        """Wait until these have arrived."""
        last = max((k for k, n in enumerate(self.reads) if n in names), default=-1)
        if last >= 0:
            self.emit(f"s_waitcnt lgkmcnt({min(len(self.reads) - 1 - last, 15)})")
            self.reads = self.reads[last + 1:]

    def a_reads(self, i):
        yield lambda: self.read(f"ds_read_b128 {self.fa(i, 0)}, %[aLo] offset:{2048 * i}", ("a", i))
        yield lambda: self.read(f"ds_read_b128 {self.fa(i, 1)}, %[aHi] offset:{2048 * i}", ("a", i))

    def a_scale(self, i):
        if self.scaled:
            yield lambda: self.read(f"ds_read_b32 {self.sm(i)}, %[aS] offset:{64 * i}", ("sa", i))

    def b_reads(self, j):
        yield lambda: self.read(f"ds_read_b128 {self.fb(j, 0)}, %[bLo] offset:{2048 * j}", ("b", j))
        yield lambda: self.read(f"ds_read_b128 {self.fb(j, 1)}, %[bHi] offset:{2048 * j}", ("b", j))

    def b_scale(self, j):
        if self.kind == "e8m0":
            yield lambda: self.read(f"ds_read_b32 {self.sn(j)}, %[bS] offset:{64 * j}", ("sb", j))
        elif self.rows:
            at = self.sn0 + 4 * j
            yield lambda: self.read(f"ds_read_b128 v[{at}:{at + 3}], %[bS] offset:{64 * j}", ("sb", j))

    def uniform_read(self, stage):
        """The wavefront's one scale of B, of the step in `stage`."""
        if self.uniform:
            yield lambda: self.read(f"ds_read_b32 {self.sn(stage)}, %[bS]", ("su", stage))

    # -- loads to LDS

    def dma(self, stage, loads):
        """Loads number `loads` (A's, B's, then the scales') of a step into `stage`."""
        for n in loads:
            if n < self.la + self.lb:
                side, k, base = ("A", n, 0) if n < self.la else ("B", n - self.la, 128 * self.bm)
                lane = f"%[{side.lower()}{'Odd' if k % 2 else 'Even'}]"
                rs = "s[60:63]" if side == "A" else "s[64:67]"

                def one(side=side, k=k, base=base, lane=lane, rs=rs):
                    self.emit(f"s_add_u32 m0, %[lds{side}], {stage * self.stride + base + 1024 * k}")
                    self.emit("s_nop 0")
                    self.emit(f"buffer_load_dwordx4 {lane}, {rs}, s{(72 if side == 'A' else 72 + self.la) + k} offen lds")
                yield one
            elif n < self.loads:
                def one():
                    if self.bytes:
                        self.emit(f"buffer_load_ubyte v{self.sv + stage}, %[gS], s[68:71], 0 offen")
                        return
                    self.emit(f"s_add_u32 m0, %[ldsS], {self.stages * self.stride + stage * self.scale_stage}")
                    self.emit("s_nop 0")
                    self.emit(f"buffer_load_{'ubyte' if self.kind == 'e8m0' else 'dword'} %[gS], s[68:71], 0 offen lds")
                yield one
            else:
                yield self.advance

    @property
    def loads(self):
        return self.la + self.lb + self.scale_loads

    def advance(self):
        """On to the next step's; past the last one's descriptors have no bytes."""
        for lo in (60, 64):
            self.emit(f"s_add_u32 s{lo}, s{lo}, 128")
            self.emit(f"s_addc_u32 s{lo + 1}, s{lo + 1}, 0")
            self.emit(f"s_sub_u32 s{lo + 2}, s{lo + 2}, 128")
        if self.scaled:
            self.emit("s_add_u32 s68, s68, s86")
            self.emit("s_addc_u32 s69, s69, s87")
        self.emit("s_sub_u32 %[left], %[left], 1")
        self.emit("s_cmp_gt_i32 %[left], 0")
        for hi in (62, 66) + ((70,) if self.scaled else ()):
            self.emit(f"s_cselect_b32 s{hi}, s{hi}, 0")

    # -- products

    def add(self, entry):
        """A result that has arrived into its sum, times its scales."""
        t, j, i, _ = entry
        at = 4 * (j * self.mt + i)
        if self.rows:
            self.need([("sa", i), ("sb", j)])
            for r in range(4):
                self.emit(f"v_mul_f32 v{t + r}, v{t + r}, {self.sm(i)}")
            for r in range(4):
                self.emit(f"v_fmac_f32 v{at + r}, v{t + r}, {self.sn(j, r)}")
        else:
            for r in range(4):
                self.emit(f"v_fmac_f32 v{at + r}, v{t + r}, {self.sm(i)}")

    def add_arrived(self):
        while self.pending and self.issued - self.pending[0][3] >= self.age:
            self.add(self.pending.pop(0))

    def mask(self, at):
        """Zero what lies past K's end of a fragment that has arrived."""
        for r in range(8):
            self.emit(f"v_and_b32 v{at + r}, v{at + r}, %[mask{'Lo' if r < 4 else 'Hi'}{r % 4}]")

    def widen(self, side, n, masked):
        """Side entries that widen a fragment, in fours."""
        raw = self.a0 + 8 * (n % self.hm) if side == "a" else self.b0 + 8 * (n % self.hn)
        to = self.wa0 + 16 * (n % self.hm) if side == "a" else self.wb0 + 16 * n

        def some(k):
            self.need([(side, n)])
            if k == 0 and masked:
                self.mask(raw)
            for r in (2 * k, 2 * k + 1):
                for high in (0, 1):
                    self.emit(f"v_cvt_scalef32_pk_f16_fp8 v{to + 2 * r + high}, v{raw + r}, 1.0"
                              + (" op_sel:[1,0,0]" if high else ""))
        return [lambda k=k: some(k) for k in range(4)]

    def quarter(self, ih, jh, stage, side, masked=()):
        """The products of halves ih of A and jh of B; `side`: what to issue
        between them, entries (first, f, tag): f after matrix instruction number
        `first` or later, and before the first that wants what `tag` names."""
        side = list(side)
        order = []
        if self.kind == "pair":  # the terms of a sum lie four apart
            for i0 in range(0, self.hm, 2):
                order += [(i, j, term) for term in range(3) for i in range(i0, min(i0 + 2, self.hm)) for j in range(self.hn)]
        elif self.wide:
            order = [(i, j, q) for i in range(self.hm) for q in range(4) for j in range(self.hn)]
        else:
            order = [(i, j, 0) for i in range(self.hm) for j in range(self.hn)]
        order = [(ih * self.hm + i, jh * self.hn + j, part) for i, j, part in order]
        total = len(order)
        fresh = set(masked)
        result = {}
        for n, (i, j, part) in enumerate(order):
            wanted = [("a", i), ("b", j)]
            while any(e[2] in wanted for e in side):
                side.pop(0)[1]()
            if self.wide:
                if part == 0:
                    result[j] = self.t0 + 4 * (self.count % 4)
                    self.count += 1
                t = result[j]
                c = f"v[{t}:{t + 3}]" if part else "0"
                self.emit(f"v_mfma_f32_16x16x32_f16 v[{t}:{t + 3}], {self.wb(j, part)}, {self.wa(i, part)}, {c}")
            else:
                self.need(wanted + ([("sa", i), ("sb", j)] if self.kind == "e8m0" else []))
                now = [x for x in wanted if x in fresh]
                fresh -= set(now)
                for name, k in now:
                    self.mask(self.a0 + 8 * (k % self.slots) if name == "a" else self.b0 + 8 * k)
                if now:
                    self.emit("s_nop 1")
                a, b = self.fa(i), self.fb(j)
                if self.kind == "e8m0":
                    self.emit(f"v_mfma_scale_f32_16x16x128_f8f6f4 {self.acc(j, i)}, {b}, {a}, {self.acc(j, i)}, "
                              f"{self.sn(j)}, {self.sm(i)} op_sel_hi:[0,0,0]")
                elif self.kind == "pair":
                    self.emit(f"v_mfma_f32_16x16x32_f16 {self.acc(j, i)}, {self.fb(j, int(part == 2))}, "
                              f"{self.fa(i, int(part == 1))}, {self.acc(j, i)}")
                else:
                    t = self.t0 + 4 * (self.count % 4)
                    self.count += 1
                    self.emit(f"v_mfma_f32_16x16x128_f8f6f4 v[{t}:{t + 3}], {b}, {a}, 0")
            self.issued += 1
            if self.after and part == (3 if self.wide else 0):
                if self.uniform and (ih, jh) in ((0, stage), (1, 1 - stage)) and j == jh * self.hn:
                    # this half's first quarter: A's scale becomes the product of both
                    self.need([("sa", i), ("su", stage)])
                    self.emit(f"v_mul_f32 {self.sm(i)}, {self.sm(i)}, {self.sn(stage)}")
                self.pending.append((t, j, i, self.issued))
            self.add_arrived()
            # the side evenly over the products, none before its time
            left = total - n - 1
            due = [e for e in side if e[0] <= n]
            take = -(-len(due) // (left + (len(due) == len(side)))) if left else len(side)
            for e in (due if left else list(side))[:take]:
                side.remove(e)
                e[1]()
        assert not side

    def meet(self, stage, under_way):
        """Loads but the newest `under_way` have arrived, those of `stage` among
        them, and all this wavefront's reads; then all wavefronts'."""
        if self.bytes:  # this thread's scale: 2^(e - 127); 0 is subnormal, 255 NaN
            sv = f"v{self.sv + stage}"
            self.emit(f"s_waitcnt vmcnt({under_way})")
            self.emit(f"v_add_u32 %[tmp], 1, {sv}")
            self.emit("v_and_b32 %[tmp], 0xff, %[tmp]")
            self.emit("v_cmp_gt_u32 vcc, 2, %[tmp]")
            self.emit("v_cndmask_b32 %[tmp], 0, %[half], vcc")
            self.emit(f"v_lshl_or_b32 %[tmp], {sv}, 23, %[tmp]")
            self.emit(f"ds_write_b32 %[wS], %[tmp] offset:{stage * self.scale_stage}")
        self.emit(f"s_waitcnt vmcnt({under_way}) lgkmcnt(0)")
        self.reads = []
        self.emit("s_barrier")

    def turn(self, stage):
        """The reads' places move to `stage` from the one before it."""
        by = 1 if stage else 1 - self.stages
        for n in ("aLo", "aHi", "bLo", "bHi"):
            self.emit(f"v_add_u32 %[{n}], {by * self.stride}, %[{n}]")
        if self.scaled:
            for n in ("aS", "bS"):
                self.emit(f"v_add_u32 %[{n}], {by * self.scale_stage}, %[{n}]")

    @staticmethod
    def entries(first, fs, tag=None):
        return [(first, f, tag) for f in fs]

    @staticmethod
    def merged(reads, loads):
        """Loads evenly among the reads."""
        out, n = [], len(loads)
        loads = list(loads)
        for k, entry in enumerate(reads):
            out.append(entry)
            while loads and (n - len(loads)) * len(reads) <= k * n:
                out.append(loads.pop(0))
        return out + loads

    def split(self):
        """How many of a step's loads start before the next step does."""
        return (self.loads * 5 + 8) // 9

    def step(self, position, last=False, masked=False):
        """A step, whose first halves have been read; last: none follows.
        masked: zero what lies past K's end, of the last step."""
        if self.wide:
            return self.wide_step(position, last, masked)
        x, y = position % 2, 1 - position % 2
        stage, after = position % self.stages, (position + 1) % self.stages
        before = (position - 1) % self.stages
        split = self.split()
        m = lambda side, h: [(side, h * n + k) for n in [self.hm if side == "a" else self.hn] for k in range(n)] if masked else []  # noqa: E731
        per = self.hn * (3 if self.kind == "pair" else 1)  # matrix instructions a fragment of A has in a quarter
        group = 2 if self.kind == "pair" else 1
        done = lambda i: per * min(i // group * group + group, self.hm) - 1  # noqa: E731  the last of them
        late = self.settled if self.after else 0

        def b_side(half):
            js = [half * self.hn + j for j in range(self.hn)]
            return ([e for j in js for e in self.entries(0, self.b_reads(j))]
                    + [e for j in js for e in self.entries(late, self.b_scale(j))])

        def a_side(half, at):
            out = []
            for i in range(self.hm):
                first = at(i)
                out += self.entries(first, self.a_reads(half * self.hm + i))
                out += self.entries(max(first, late), self.a_scale(half * self.hm + i))
            return out

        side = b_side(y)
        if self.slots == self.mt:  # room beside the first half
            side += a_side(1, lambda i: 0)
        if not last:
            side = self.merged(side, self.entries(0, self.dma(before, range(split, self.loads + 1))))
        self.quarter(0, x, x, side, m("a", 0) + m("b", x))
        self.quarter(0, y, x, a_side(1, done) if self.slots < self.mt else [], m("b", y))
        self.quarter(1, y, x, [], m("a", 1))
        side = []
        if not last:
            self.meet(after, self.loads * (self.stages - 2))
            self.turn(after)
            side = b_side(y) + self.entries(0, self.uniform_read(y))
            side += a_side(0, done if self.slots < self.mt else lambda i: 0)
            side = self.merged(side, self.entries(0, self.dma(stage, range(split))))
        self.quarter(1, x, x, side)

    def wide_step(self, position, last, masked):
        """At its begin the first half of B and A's first fragment are widened,
        the rest of A's first half has been read.  masked: the last step is this
        one, or the next (what is widened here of it)."""
        x, y = position % 2, 1 - position % 2
        stage, after = position % self.stages, (position + 1) % self.stages
        before = (position - 1) % self.stages
        split = self.split()
        half = 4 * self.hn  # matrix instructions a fragment of A has in a quarter
        assert self.hm == 2
        bs = lambda h: [h * self.hn + j for j in range(self.hn)]  # noqa: E731

        side = self.entries(0, self.widen("a", 1, masked and last), ("a", 1))
        for j in bs(y):
            side += self.entries(0, self.b_reads(j))
        side += self.entries(0, self.a_reads(2)) + self.entries(0, self.a_reads(3))
        for i in (2, 3):
            side += self.entries(self.settled, self.a_scale(i))
        for j in bs(y):
            side += self.entries(self.settled, self.b_scale(j))
        if not last:
            side = self.merged(side, self.entries(0, self.dma(before, range(split, self.loads + 1))))
        for j in bs(y):
            side += self.entries(half, self.widen("b", j, masked and last), ("b", j))
        self.quarter(0, x, x, side)
        self.quarter(0, y, x, self.entries(half - 1, self.widen("a", 2, masked and last), ("a", 2)))
        side = self.entries(0, self.widen("a", 3, masked and last), ("a", 3))
        if not last:
            self.meet(after, self.loads * (self.stages - 2))
            self.turn(after)
            side += self.entries(0, self.a_reads(0)) + [e for j in bs(y) for e in self.entries(0, self.b_reads(j))]
            side += self.entries(0, self.a_reads(1)) + self.entries(0, self.uniform_read(y))
            for i in (0, 1):
                side += self.entries(self.settled, self.a_scale(i))
            side = self.merged(side, self.entries(0, self.dma(stage, range(split))))
        self.quarter(1, y, x, side)
        side = []
        if not last:
            for j in bs(y):
                side += self.entries(0, self.widen("b", j, masked), ("b", j))
                side += self.entries(self.settled, self.b_scale(j))
            side += self.entries(half - 1, self.widen("a", 0, masked), ("a", 0))
        self.quarter(1, x, x, side)

    def start(self, position):
        """The loads of the first steps, the very first in `position`."""
        for ahead in range(self.stages - 1):
            for f in self.dma((position + ahead) % self.stages, range(self.loads + 1)):
                f()
        for f in self.dma((position - 1) % self.stages, range(self.split())):
            f()
        self.first_meet = (position % self.stages, self.loads * (self.stages - 2) + self.split())

    def first_reads(self, x):
        for f in self.uniform_read(x):
            f()
        for i in range(self.hm):
            for f in list(self.a_reads(i)) + list(self.a_scale(i)):
                f()
        for j in range(x * self.hn, (x + 1) * self.hn):
            for f in list(self.b_reads(j)) + list(self.b_scale(j)):
                f()
        self.emit("s_waitcnt lgkmcnt(0)")
        self.reads = []

    def prime(self, x, masked):
        """What of the first step is widened where it begins."""
        if self.wide:
            for f in [f for j in range(x * self.hn, (x + 1) * self.hn) for f in self.widen("b", j, masked)] + self.widen("a", 0, masked):
                f()

    def state(self):
        """What is under way and pending, counted from here."""
        return list(self.reads), [(t, j, i, n - self.issued) for t, j, i, n in self.pending], self.count % 4

    def enter(self, state):
        self.reads, self.pending, self.count = list(state[0]), list(state[1]), state[2]
        self.issued = 0

    def text(self):
        """The whole loop: %[first] the position of the first step, %[turns] the
        times that the last position but one is passed before the last two
        steps, %[left] the number of steps."""
        # what is under way and pending where a step begins: as the step before leaves it
        probe = Loop(self.kind, self.mt, self.nt, self.wm, self.wn, self.stages)
        begin = {}
        for position in list(range(self.positions)) * 2:
            state = probe.state()
            assert position not in begin or position == 0 or begin[position] == state
            begin[position] = state
            probe.step(position)
        assert begin[0] == probe.state() and all(begin[p] == begin[p % 2] for p in begin)
        top = self.positions - 1

        def take(position, label, **how):
            self.emit(f".Lnt_{label}_%=:")
            self.enter(begin[position])
            self.step(position, **how)
            assert how.get("last") or self.state() == begin[(position + 1) % 2]

        self.emit("s_mov_b32 s72, %[oA]")
        for k in range(1, self.la):
            self.emit(f"s_add_u32 s{72 + k}, s{71 + k}, %[eA]")
        self.emit(f"s_mov_b32 s{72 + self.la}, %[oB]")
        for k in range(1, self.lb):
            self.emit(f"s_add_u32 s{72 + self.la + k}, s{71 + self.la + k}, %[eB]")
        for stage in range(1, self.stages):
            for position in range(stage, self.positions, self.stages):
                self.emit(f"s_cmp_eq_u32 %[first], {position}")
                self.emit(f"s_cbranch_scc1 .Lnt_start{stage}_%=")
        for stage in range(self.stages):
            if stage:
                self.emit(f".Lnt_start{stage}_%=:")
            self.start(stage)
            if self.bytes:  # only this place knows which register the bytes are in
                self.zeros()
                self.meet(*self.first_meet)
            if stage < self.stages - 1:
                self.emit("s_branch .Lnt_started_%=")
        self.emit(".Lnt_started_%=:")
        if not self.bytes:
            self.zeros()
            self.meet(*self.first_meet)
        self.emit("s_bitcmp1_b32 %[first], 0")
        self.emit("s_cbranch_scc1 .Lnt_odd_%=")
        self.first_reads(0)
        self.prime(0, False)
        self.jump(range(0, top - 1, 2))
        self.emit("s_branch .Lnt_check_%=")
        self.emit(".Lnt_odd_%=:")
        self.first_reads(1)
        self.emit(f"s_cmp_eq_u32 %[first], {top}")
        self.emit("s_cbranch_scc1 .Lnt_top_%=")
        self.prime(1, False)
        self.jump(range(1, top - 1, 2))
        if self.positions > 2:
            self.emit("s_branch .Lnt_check_%=")
        # the first position is the last when there is one step, or one over whole turns
        self.emit(".Lnt_top_%=:")
        self.emit("s_cmp_eq_u32 %[single], 1")
        self.emit("s_cbranch_scc1 .Lnt_single_%=")
        self.prime(1, False)
        take(top, "turn")
        for position in range(top - 1):
            take(position, position)
        self.emit(".Lnt_check_%=:")
        self.emit("s_cmp_eq_u32 %[turns], 0")
        self.emit("s_cbranch_scc1 .Lnt_next_%=")
        self.emit("s_sub_u32 %[turns], %[turns], 1")
        take(top - 1, "before")
        self.emit("s_branch .Lnt_turn_%=")
        take(top - 1, "next", masked=self.wide)
        self.emit("s_branch .Lnt_last_%=")
        self.emit(".Lnt_single_%=:")
        self.prime(1, True)
        self.emit(".Lnt_last_%=:")
        if self.scaled and not self.wide:
            self.emit("s_cmp_lg_u32 %[partial], 0")
            self.emit("s_cbranch_scc1 .Lnt_masked_%=")
        take(top, "whole", last=True, masked=self.wide)
        self.drain()
        if self.scaled and not self.wide:
            self.emit("s_branch .Lnt_end_%=")
            take(top, "masked", last=True, masked=True)
            self.drain()
            self.emit(".Lnt_end_%=:")
        return self.lines

    def zeros(self):
        for n in list(range(4 * self.mt * self.nt)) + list(range(self.t0, self.sv)):
            self.emit(f"v_mov_b32 v{n}, 0")

    def jump(self, positions):
        for position in positions:
            self.emit(f"s_cmp_eq_u32 %[first], {position}")
            self.emit(f"s_cbranch_scc1 .Lnt_{position}_%=")

    def drain(self):
        self.emit("s_waitcnt vmcnt(0) lgkmcnt(0)")
        self.reads = []
        self.emit("s_nop 15")
        self.emit("s_nop 7")
        for p in self.pending:
            self.add(p)
        self.pending = []

    def name(self):
        return f"{self.kind}_{self.bm}x{self.bn}"


LOOPS = [
    ("e8m0", 8, 4, 2, 4, 2), ("f32u", 8, 4, 2, 4, 2), ("f32n", 8, 4, 2, 4, 2),
    ("e8m0", 4, 4, 4, 2, 3), ("f32u", 4, 4, 4, 2, 3), ("f32n", 4, 4, 4, 2, 3),
    ("w32u", 4, 4, 2, 2, 2), ("w32n", 4, 4, 2, 2, 2), ("w8u", 4, 4, 2, 2, 2), ("w8n", 4, 4, 2, 2, 2),
    ("pair", 8, 4, 2, 4, 2), ("pair", 6, 6, 2, 2, 3), ("pair", 4, 2, 2, 4, 4),
]


def generate() -> str:
    out = ["// Generated by gen_nt_loop.py (the K loops of nt_loop.h); do not edit."]
    for args in LOOPS:
        loop = Loop(*args)
        name = loop.name()
        text = loop.text()
        out.append(f"#define NT_LOOP_{name} \\")
        out += [f'  "{line}\\n" \\' for line in text]
        out.append('  ""')
        spare = range(4 * loop.mt * loop.nt, loop.registers)
        out.append(f"#define NT_CLOBBERS_{name} " + ", ".join(f'"v{n}"' for n in spare)
                   + ", " + ", ".join(f'"s{72 + n}"' for n in range(loop.la + loop.lb)) + (', "vcc"' if loop.bytes else ""))
    return "\n".join(out) + "\n"


if __name__ == "__main__":
    with open(OUT, "w") as f:
        f.write(generate())
