"""What follows a step of drafted tokens: lengths taken back over a page's edge, their pages returned to the list, and accepted
drafts that do not lie together written again.  Bounds as in test_gpu_prompt_attn."""
import random

import pytest
import torch

from paged_reference import PAGE, blocks, dense_reference
from test_gpu_many_tokens_step import Loop, msa  # noqa: F401
from test_gpu_prompt_attn import check, reference

pytestmark = pytest.mark.gpu


class Drafts(Loop):
    def take_back(self, lens):
        """Shortens the sequences, as the header tells a caller to."""
        back = [self.table[s, b].item() for s, (a, n) in enumerate(zip(self.lens, lens)) for b in range(blocks(n), blocks(a))]
        at = self.taken.item()
        if back:
            self.free[at - len(back):at] = torch.tensor(back, dtype=torch.int32, device="cuda")
            self.taken -= len(back)
        self.lens = list(lens)
        self.device_lens.copy_(torch.tensor(lens, dtype=torch.int32))

    def no_page_is_lost(self):
        held = [p for s, n in enumerate(self.lens) for p in self.table[s, :blocks(n)].tolist()]
        left = self.free[self.taken.item():].tolist()
        assert self.taken.item() == len(held) and sorted(held + left) == list(range(self.k.shape[0] // PAGE))


def next_rows(lp, seen):
    """grow() that also keeps the step's k and v."""
    rows = lp.rows

    def keep(n):
        seen[:] = rows(n)
        return tuple(seen)
    lp.rows = keep


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("first,new,left", [(120, 10, 127), (120, 10, 128), (127, 3, 127), (127, 3, 128), (128, 2, 128), (250, 300, 251), (1, 127, 1)])
def test_lengths_taken_back(msa, fp8, first, new, left):
    """Also to a length that ends with its block, and over several blocks; then steps of one token and a chunk."""
    lp = Drafts(msa, 2, 16, 2, fp8, pages=40)
    lp.grow([first, 77])
    lp.grow([new, 1])
    lp.take_back([left, 77])
    lp.no_page_is_lost()
    prefill = msa.msa_dense_attn_prefill_paged_fp8 if fp8 else msa.msa_dense_attn_prefill_paged
    decode = msa.msa_dense_attn_decode_paged_fp8 if fp8 else msa.msa_dense_attn_decode_paged
    for step in ([1, 1], [1, 1], [140, 60]):
        prob, q = lp.grow(step)
        lp.no_page_is_lost()
        caches = (lp.k, lp.v, *lp.scales(), lp.table)
        check(prefill(prob, q, *caches), reference(step, lp.lens, lp.key_rows(), q, lp.k, lp.v, lp.ks, lp.vs, 0.0, None), f"{step}")
        if step == [1, 1]:
            o, lse = decode(prob, q, *caches)
            ro, rl, _, to, tl, _ = dense_reference(lp.lens, lp.table, q, lp.k, lp.v, lp.ks, lp.vs)
            assert ((o.double() - ro).abs() <= to).all() and ((lse.double() - rl).abs() <= tl).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_speculative_loop(msa, fp8):
    """Trees step after step, a path of each accepted: the pool holds what the sequences need, the cache what was accepted."""
    lp, rng, S = Drafts(msa, 3, 16, 2, fp8, pages=60, seed=9), random.Random(2), 3
    tree = msa.msa_tree_attn_paged_fp8 if fp8 else msa.msa_tree_attn_paged
    append = msa.msa_append_paged_fp8 if fp8 else msa.msa_append_paged
    kept = []   # the rows that the cache has to hold: (k, v) of each sequence
    rows = []
    next_rows(lp, rows)
    lp.grow([120, 250, 7])
    for a, b in zip((0, 120, 370), (120, 370, 377)):
        kept.append([rows[1][a:b], rows[2][a:b]])
    for step in range(12):
        new, before = [rng.randint(1, 9) for _ in range(S)], lp.lens
        prob, q = lp.grow(new)
        parents = [[-1] + [rng.randint(0, i - 1) for i in range(1, n)] for n in new]
        see = []
        for par in parents:
            m = torch.eye(len(par), dtype=torch.bool)
            for i, a in enumerate(par):
                if a >= 0:
                    m[i] |= m[a]
            see.append(m)
        bits = torch.cat([(m.long() << torch.arange(m.shape[1])).sum(1) for m in see]).to(torch.int32).view(-1, 1).cuda()
        got = tree(prob, q, lp.k, lp.v, *lp.scales(), lp.table, bits)
        check(got, reference(new, lp.lens, lp.key_rows(), q, lp.k, lp.v, lp.ks, lp.vs, 0.0, see), f"step {step}")
        # the path to some draft is accepted
        slots = torch.cat([r[a:] for r, a in zip(lp.key_rows(), before)]).cuda()
        at, src, dst, lens = 0, [], [], []
        for s, (n, m) in enumerate(zip(new, see)):
            path = [j for j, b in enumerate(m[rng.randrange(n)].tolist()) if b]
            src += [at + j for j in path]
            dst += list(range(at, at + len(path)))
            lens.append(before[s] + len(path))
            kept[s] = [torch.cat([x, y[[at + j for j in path]]]) for x, y in zip(kept[s], rows[1:])]
            at += n
        append(rows[1][src], rows[2][src], slots[dst], lp.k, lp.v, *lp.scales())
        lp.take_back(lens)
        lp.no_page_is_lost()
    for s, r in enumerate(lp.key_rows()):
        r = r.cuda()
        for x, cache, scale in ((kept[s][0], lp.k, lp.ks), (kept[s][1], lp.v, lp.vs)):
            if not fp8:
                assert torch.equal(cache[r], x)
                continue
            held = cache[r].view(torch.float8_e4m3fn).float() * scale[r // PAGE][:, :, None]
            # a code is off by half a step, 2^-4 of the value, and below 2^-6 by 2^-10, of the scale; a row is rounded again each time
            # that its page's scale grows, at most by so much at each
            assert ((held - x.float()).abs() <= 12 * (2.0 ** -4 * x.float().abs() + 2.0 ** -10 * scale[r // PAGE][:, :, None])).all()
