"""A serving run: prompts numbered and written, trees of drafted tokens attended to and
their accepted paths kept, single tokens and chunks over a window, pages taken and given
back in between -- against the tokens themselves, kept on the host."""
import random

import pytest
import torch

from decode_attention_paged_pa_gb300 import binding
from view_testutil import ancestors, attend64, tree_parents

pytestmark = pytest.mark.gpu
DEV = "cuda"
S, H, KH, D, BS, MB, NB, LAYERS = 5, 8, 2, 64, 16, 24, 100, 2
SCALES = dict(k_scale=0.05, v_scale=0.07)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Server:
    """Requests on the device, and what their caches should hold on the host: per layer
    and request, keys and values [tokens, KH, D] as the cache keeps them."""

    def __init__(self, dtype, e4m3, seed):
        self.dtype, self.e4m3 = dtype, e4m3
        self.g, self.r = torch.Generator().manual_seed(seed), random.Random(seed)
        ct = torch.uint8 if e4m3 else dtype
        x = 16 if e4m3 else 8
        poison = 0x7F if e4m3 else float("nan")
        self.keys = [torch.full((NB, KH, D // x, BS, x), poison, dtype=ct, device=DEV) for _ in range(LAYERS)]
        self.values = [torch.full((NB, KH, D, BS), poison, dtype=ct, device=DEV) for _ in range(LAYERS)]
        self.tables = torch.full((S, MB), -1, dtype=torch.int32, device=DEV)
        self.lens, self.refs = i32([0] * S), i32([0] * NB)
        self.want = [[[torch.zeros((0, KH, D), dtype=ct) for _ in range(2)] for _ in range(S)] for _ in range(LAYERS)]

    def ok(self, ws):
        assert binding.device_status(ws) == binding.PA_OK

    def rows(self, *shape):
        return torch.randn(shape, generator=self.g).to(self.dtype)

    def kept(self, x, scale):
        return (x.float() / torch.tensor(scale)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if self.e4m3 else x

    def resize(self, new):
        self.ok(binding.pa_pages_resize(self.tables, self.lens, i32(new), self.refs, self.keys + self.values, BS))
        assert self.lens.tolist() == new

    def add(self, counts, room=7):
        """New tokens of every request: their pages, slots, and rows in every layer."""
        self.resize([L + c for L, c in zip(self.lens.tolist(), counts)])
        total = sum(counts)
        N = total + room
        slots = torch.empty((N,), dtype=torch.int64, device=DEV)
        positions, ids, cu = i32([9] * N), i32([9] * N), i32([9] * (S + 1))
        self.ok(binding.pa_pages_slots(slots, positions, ids, cu, self.tables, self.lens, i32(counts), BS))
        assert positions[:total].tolist() == [L - c + i for L, c in zip(self.lens.tolist(), counts) for i in range(c)]
        assert ids[:total].tolist() == [s for s, c in enumerate(counts) for _ in range(c)]
        for layer in range(LAYERS):
            qkv = self.rows(N, H + 2 * KH, D)  # (rows as a projection leaves them)
            d = qkv.to(DEV)
            more = SCALES if self.e4m3 else {}
            self.ok(binding.pa_cache_write(self.keys[layer], self.values[layer], d[:, H:H + KH], d[:, H + KH:], slots, **more))
            at = 0
            for s, c in enumerate(counts):
                new = self.kept(qkv[at:at + c, H:H + KH], SCALES["k_scale"]), self.kept(qkv[at:at + c, H + KH:], SCALES["v_scale"])
                self.want[layer][s] = [torch.cat([a, b]) for a, b in zip(self.want[layer][s], new)]
                at += c

    def check(self, layer, q, out, window, sinks, see=None):
        """Against 64-bit attention over the host's tokens, in pages of their own."""
        x = 16 if self.e4m3 else 8
        kc = torch.zeros((S * MB, KH, D // x, BS, x), dtype=self.keys[0].dtype)
        vc = torch.zeros((S * MB, KH, D, BS), dtype=kc.dtype)
        for s in range(S):
            k, v = self.want[layer][s]
            assert k.shape[0] == int(self.lens[s])
            t = torch.arange(k.shape[0])
            kc[s * MB + t // BS, :, :, t % BS] = k.view(-1, KH, D // x, x)
            vc[s * MB + t // BS, :, :, t % BS] = v
        tables = torch.arange(S * MB).view(S, MB)
        more = SCALES if self.e4m3 else {}
        ref, _, bound = attend64(q, kc, vc, tables, self.lens.tolist(), 0.125, window, sinks, see, **more)
        err = (out.cpu().view(q.shape).double() - ref).abs()
        assert bool((err <= bound).all()), f"worst excess {float((err - bound).max()):.3e}"

    def window(self, n, window, sinks):
        self.add([n] * S)
        for layer in range(LAYERS):
            q = self.rows(S, n, H, D)
            d = q.to(DEV) if n > 1 else q[:, 0].to(DEV)
            out = torch.full_like(d, float("nan"))
            call, more = (binding.pa_decode_v2_window_fp8, SCALES) if self.e4m3 else (binding.pa_decode_v2_window, {})
            self.ok(call(out, d, self.keys[layer], self.values[layer], self.tables, self.lens, 0.125, window, sinks,
                         partition_size=64, **more))
            self.check(layer, q, out, window, sinks)

    def tree(self, n, window):
        before = self.lens.tolist()
        parents = [tree_parents(self.r.randrange(1 << 20), n, self.r.randint(1, n)) for _ in range(S)]
        see = torch.stack([ancestors(p) for p in parents])
        self.add([n] * S)
        masks, positions = torch.zeros((S, n, (n + 31) // 32), dtype=torch.int32, device=DEV), i32([[0] * n] * S)
        self.ok(binding.pa_tree_masks(masks, positions, i32(parents), self.lens))
        for layer in range(LAYERS):
            w = window if layer else 0  # (the first layer sees everything)
            q = self.rows(S, n, H, D)
            d = q.to(DEV)
            out = torch.full_like(d, float("nan"))
            call, more = (binding.pa_decode_v2_tree_fp8, SCALES) if self.e4m3 else (binding.pa_decode_v2_tree, {})
            self.ok(call(out, d, self.keys[layer], self.values[layer], self.tables, self.lens, masks, 0.125, window=w, sinks=2,
                         partition_size=64, **more))
            self.check(layer, q, out, w, 2, see)
        # A path down each tree is accepted: the ancestors of one of its nodes, or nothing.
        paths = [see[s, self.r.randrange(n)].nonzero().flatten().tolist() for s in range(S)]
        paths[self.r.randrange(S)] = []
        accepted = i32([p + [-7] * (n - len(p)) for p in paths])
        new_lens = i32([0] * S)
        self.ok(binding.pa_tree_accept(new_lens, self.keys, self.values, self.tables, self.lens, accepted,
                                       i32([len(p) for p in paths]), n))
        new = [b + len(p) for b, p in zip(before, paths)]
        assert new_lens.tolist() == new
        for layer in self.want:
            for s, p in enumerate(paths):
                layer[s] = [torch.cat([t[:before[s]], t[before[s]:][p]]) for t in layer[s]]
        self.resize(new)


@pytest.mark.parametrize("dtype,e4m3", [(torch.float16, False), (torch.bfloat16, False), (torch.bfloat16, True)])
def test_run(dtype, e4m3):
    sv = Server(dtype, e4m3, 3)
    sv.add([40, 1, 17, 0, 64])
    for n, window in ((7, 20), (1, 4), (33, 33)):
        sv.tree(n, window)
        sv.window(1, 30, 4)
    sv.window(20, 25, 3)
    # One request ends and another takes its row.
    lens = sv.lens.tolist()
    lens[0] = 0
    sv.resize(lens)
    for layer in sv.want:
        layer[0] = [t[:0] for t in layer[0]]
    sv.add([50, 0, 0, 3, 0])
    sv.tree(16, 64)
    sv.window(1, 1000, 0)
    used = int((sv.refs > 0).sum())
    assert used == sum(-(-L // BS) for L in sv.lens.tolist())
