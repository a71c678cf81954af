"""Helpers of the GPU tests around the recurrent layers: packs of requests on the device."""
import numpy as np

from packed_linear_attention_gb300 import gdn

from gpu_util import torch_cuda

IO = {"bf16": (gdn.GDN_BF16, 2.0 ** -8), "f32": (gdn.GDN_F32, 2.0 ** -24)}


def dtype(io):
    torch = torch_cuda()
    return torch.bfloat16 if io == "bf16" else torch.float32


def up(x, io="f32"):
    torch = torch_cuda()
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda().to(dtype(io))


def i32(x):
    torch = torch_cuda()
    return torch.tensor(np.asarray(x).tolist(), dtype=torch.int32, device="cuda")


def num(t):
    return t.detach().double().cpu().numpy()


def rows(rng, n, ch, io, gap=8, scale=1.0):
    """[n, ch] as a column range of a wider array, on 16-byte boundaries."""
    wide = -(-ch // 8) * 8 + gap
    return up(scale * rng.standard_normal((n, wide)), io)[:, :ch]


def empty_rows(n, ch, io, fill=7.0):
    torch = torch_cuda()
    return torch.full((n, -(-ch // 8) * 8), fill, dtype=dtype(io), device="cuda")[:, :ch]


class Pack:
    """Requests of the given lengths, with slots in a shuffled order and checkpoints anywhere."""

    def __init__(self, rng, lens, spare_rows=3, spare_slots=2, ckpt=True, max_len=None):
        self.lens = list(lens)
        b = len(lens)
        self.cu = np.concatenate([[0], np.cumsum(lens)]).astype(int)
        self.tokens = int(self.cu[-1]) + spare_rows
        self.slots = b + spare_slots
        self.slot = rng.permutation(self.slots)[:b]
        self.zero = rng.integers(0, 2, b)
        self.pos = [sorted(rng.choice(np.arange(1, n + 1), min(n, int(k)), replace=False).tolist())
                    if ckpt and n else [] for n, k in zip(lens, rng.integers(0, 4, b))]
        self.ckpt_cu = np.concatenate([[0], np.cumsum([len(p) for p in self.pos])]).astype(int)
        self.flat = [p for q in self.pos for p in q]
        self.num_ckpt = len(self.flat)
        self.max_len = max(lens) if max_len is None else max_len
        self.keep = [i32(self.cu), i32(self.slot), i32(self.zero), i32(self.ckpt_cu),
                     i32(self.flat + [0])]
        cu, slot, zero, ckpt_cu, pos = self.keep
        self.requests = gdn.make_requests(cu, self.tokens, self.max_len, self.slots, slot_idx=slot,
                                          start_zero=zero, ckpt_cu=ckpt_cu, ckpt_pos=pos,
                                          num_ckpt=self.num_ckpt)
