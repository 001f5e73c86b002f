"""The 4-bit cache and the page operators together, as a server uses them:
prompts come in, are decoded, forked and verified with draft tokens, sequences
end, the pool is compacted.  A plain model keeps every sequence's quantised
tokens as a list; after every step the attention over the paged cache has to
agree with attention over that list, the rows read back with its values, and
the block counts with the tables."""
import math

import pytest
import torch

from decode_attention_paged_pa_gb300 import binding
from kv4_testutil import attend64, pack_records, quantise64

pytestmark = pytest.mark.gpu

KH, H, D, BS, MB, NB = 2, 8, 64, 16, 12, 90


class Server:
    def __init__(self, dtype, layers=2):
        self.dev = torch.device("cuda")
        self.dtype = dtype
        self.g = torch.Generator().manual_seed(5)
        self.caches = [torch.randint(0, 256, (NB, KH, binding.kv4_block_bytes(D, BS)), dtype=torch.uint8,
                                     generator=self.g).to(self.dev) for _ in range(layers)]
        self.rows = 6
        self.tables = torch.zeros((self.rows, MB), dtype=torch.int32, device=self.dev)
        self.lens = torch.zeros(self.rows, dtype=torch.int32, device=self.dev)
        self.refs = torch.zeros(NB, dtype=torch.int32, device=self.dev)
        self.model = [[[] for _ in range(self.rows)] for _ in range(layers)]  # per token (codes k, v, params)

    def i32(self, v):
        return torch.tensor(v, dtype=torch.int32, device=self.dev)

    def ok(self, ws):
        assert binding.device_status(ws) == binding.PA_OK

    def resize(self, new):
        self.ok(binding.pa_pages_resize(self.tables, self.lens, self.i32(new), self.refs, self.caches, BS))
        for layer in self.model:
            for s, n in enumerate(new):
                del layer[s][n:]

    def append(self, new):
        """new[s] tokens more for each sequence: room first, then the tokens of every layer."""
        self.resize([len(t) + n for t, n in zip(self.model[0], new)])
        cu = self.i32([sum(new[:s]) for s in range(len(new) + 1)])
        for cache, layer in zip(self.caches, self.model):
            k, v = ((torch.randn((sum(new), KH, D), generator=self.g) + 0.3).to(self.dtype) for _ in range(2))
            self.ok(binding.pa_kv4_append(cache, k.to(self.dev), v.to(self.dev), self.tables, self.lens, cu_tokens=cu))
            (kc, ks, kz), (vc, vs, vz) = quantise64(k), quantise64(v)
            par = torch.cat([ks, kz, vs, vz], -1).to(self.dtype)
            row = 0
            for s, n in enumerate(new):
                for _ in range(n):
                    layer[s].append((kc[row].to(torch.uint8), vc[row].to(torch.uint8), par[row]))
                    row += 1

    def dense(self, layer):
        """The model's tokens as a cache of its own: block b of sequence s at s * MB + b."""
        kc = torch.zeros((self.rows * MB, KH, BS, D), dtype=torch.uint8)
        vc, par = kc.clone(), torch.zeros((self.rows * MB, KH, BS, 4), dtype=self.dtype)
        for s, tokens in enumerate(layer):
            for t, (k, v, p) in enumerate(tokens):
                at = (s * MB + t // BS, slice(None), t % BS)
                kc[at], vc[at], par[at] = k, v, p
        return pack_records(kc, vc, par), torch.arange(self.rows * MB, dtype=torch.int32).view(self.rows, MB)

    def check(self, q_len=1):
        lens = [len(t) for t in self.model[0]]
        assert self.lens.tolist() == lens
        # every block that a row holds is counted, no other
        want = [0] * NB
        for s, n in enumerate(lens):
            for b in self.tables[s, : -(-n // BS)].tolist():
                want[b] += 1
        assert self.refs.tolist() == want
        for cache, layer in zip(self.caches, self.model):
            if min(lens) >= q_len or q_len == 1:
                shape = (self.rows, H, D) if q_len == 1 else (self.rows, q_len, H, D)
                q = torch.randn(shape, generator=self.g).to(self.dtype)
                out = torch.empty_like(q, device=self.dev)
                call = binding.pa_decode_v2_kv4 if q_len == 1 else binding.pa_decode_v2_mq_kv4
                self.ok(call(out, q.to(self.dev), cache, self.tables, self.lens, 1 / math.sqrt(D), partition_size=64))
                rec, bt = self.dense(layer)
                ref, bound, _, _ = attend64(q, rec, bt, torch.tensor(lens), 1 / math.sqrt(D), self.dtype)
                assert bool(((out.cpu().double() - ref).abs() <= bound).all())
            total = sum(lens)
            k, v = (torch.empty((total, KH, D), dtype=self.dtype, device=self.dev) for _ in range(2))
            cu = self.i32([sum(lens[:s]) for s in range(len(lens) + 1)])
            self.ok(binding.pa_kv4_gather(k, v, cache, self.tables, self.lens, cu_tokens=cu))
            tokens = [t for seq in layer for t in seq]
            for got, i in ((k.cpu().double(), 0), (v.cpu().double(), 1)):
                if not tokens:
                    continue
                c = torch.stack([t[i] for t in tokens]).double()
                p = torch.stack([t[2] for t in tokens]).double()
                ref = c * p[..., 2 * i:2 * i + 1] + p[..., 2 * i + 1:2 * i + 2]
                half = torch.finfo(self.dtype).eps / 2
                assert bool(((got - ref).abs() <= half * ref.abs() * 1.01 + 2.0 ** -25).all())

    def fork(self, parents):
        """The batch becomes forks of its own rows (-1: an empty row); the old rows are freed."""
        out = torch.zeros_like(self.tables)
        lens = torch.zeros_like(self.lens)
        self.ok(binding.pa_pages_fork(out, lens, self.tables, self.lens, self.i32(parents), self.refs, self.caches, BS))
        old_t, old_l = self.tables, self.lens
        self.ok(binding.pa_pages_resize(old_t, old_l, torch.zeros_like(old_l), self.refs, self.caches, BS))
        self.tables, self.lens = out, lens
        self.model = [[list(layer[p]) if p >= 0 else [] for p in parents] for layer in self.model]

    def compact(self):
        self.ok(binding.pa_pages_compact(self.tables, self.lens, self.refs, self.caches, BS))
        used = int((self.refs > 0).sum())
        assert bool((self.refs[:used] > 0).all())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
def test_serving(dtype):
    s = Server(dtype)
    s.check()
    s.append([33, 5, 100, 0, 16, 17])          # prompts
    s.check()
    for _ in range(3):                         # steps
        s.append([1, 1, 1, 0, 1, 1])
    s.check()
    s.fork([2, 2, 0, 0, 5, -1])                # beams: shared full pages, copies of the open ones
    s.check()
    s.append([1, 1, 1, 1, 1, 40])              # they go on apart; a new prompt
    s.check()
    s.append([4] * 6)                          # drafts, verified at once
    s.check(q_len=4)
    n = [len(t) for t in s.model[0]]
    s.resize([n[0] - 3, n[1], n[2] - 1, 0, n[4] - 4, n[5] - 2])   # some refused, one sequence ends
    s.check()
    s.compact()
    s.check()
    s.append([1, 20, 1, 60, 1, 1])
    s.check()
    s.resize([60, 64, 5, 10, 0, 16])           # cut back, some of it into shared pages
    s.check()
    s.append([2, 2, 2, 2, 0, 2])
    s.check()
    s.fork([0, 0, 0, 1, 1, 1])
    s.append([3, 2, 1, 3, 2, 1])
    s.compact()
    s.check(q_len=2)
    s.resize([0] * 6)
    s.check()
    assert int(s.refs.sum()) == 0
