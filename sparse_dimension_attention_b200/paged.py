"""Device buffers of the paged 8-bit cache and the rotation table, as PyTorch tensors.

The objects own their tensors and the descriptors that point at them; all
computation on the buffers happens in the CUDA library.  Lengths stay with the
caller, who also writes block_table.
"""
from __future__ import annotations

import torch

from . import abi


class AquaPagedCache:
    """Pages of projected keys and values in e4m3, their scales, and the block table.

    k_pages [n_pages, Hkv, d_store, page_size] and v_pages [n_pages, Hkv,
    page_size, d] (uint8 codes; .view(torch.float8_e4m3fn) reads them), k_scale
    and v_scale [n_pages, Hkv] f32, block_table [B, max_pages] int32 (-1: unset).
    """

    def __init__(self, B: int, Hkv: int, n_pages: int, max_pages: int, page_size: int = 64, d: int = 128,
                 d_store: int | None = None, device="cuda"):
        d_store = d if d_store is None else d_store
        self._adopt(torch.zeros((n_pages, Hkv, d_store, page_size), dtype=torch.uint8, device=device),
                    torch.zeros((n_pages, Hkv, page_size, d), dtype=torch.uint8, device=device),
                    torch.ones((n_pages, Hkv), dtype=torch.float32, device=device),
                    torch.ones((n_pages, Hkv), dtype=torch.float32, device=device),
                    torch.full((B, max_pages), -1, dtype=torch.int32, device=device))

    @classmethod
    def from_buffers(cls, k_pages, v_pages, k_scale, v_scale, block_table) -> "AquaPagedCache":
        """A cache over tensors the caller allocated (they are kept alive, not copied)."""
        self = cls.__new__(cls)
        self._adopt(k_pages, v_pages, k_scale, v_scale, block_table)
        return self

    def _adopt(self, k_pages, v_pages, k_scale, v_scale, block_table) -> None:
        n_pages, Hkv, d_store, page_size = k_pages.shape
        d = v_pages.shape[-1]
        B, max_pages = block_table.shape
        for t, shape, dtype in ((k_pages, (n_pages, Hkv, d_store, page_size), torch.uint8),
                                (v_pages, (n_pages, Hkv, page_size, d), torch.uint8),
                                (k_scale, (n_pages, Hkv), torch.float32), (v_scale, (n_pages, Hkv), torch.float32),
                                (block_table, (B, max_pages), torch.int32)):
            if t.shape != shape or t.dtype != dtype or not t.is_contiguous() or t.device != k_pages.device:
                raise abi.AquaError(abi.AQUA_ERR_ARG, f"paged cache buffer {tuple(t.shape)} {t.dtype} on {t.device}: "
                                                      f"expected contiguous {shape} {dtype} on {k_pages.device}")
        self.B, self.Hkv, self.d, self.d_store = B, Hkv, d, d_store
        self.n_pages, self.max_pages, self.page_size = n_pages, max_pages, page_size
        self.k_pages, self.v_pages, self.k_scale, self.v_scale = k_pages, v_pages, k_scale, v_scale
        self.block_table = block_table
        self.ctrl = torch.zeros((abi.AQUA_CTRL_WORDS,), dtype=torch.int32, device=k_pages.device)
        self.desc = abi.aqua_paged_cache(
            k_pages.data_ptr(), v_pages.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(),
            self.ctrl.data_ptr(), B, Hkv, d, d_store, page_size, n_pages, max_pages, abi.AQUA_E4M3)
        self.desc.device = k_pages.get_device()


class AquaRope:
    """Position rotation: cos_sin [n_pos, rot_dim] f32, the cosines of each position's angles, then the sines."""

    def __init__(self, cos_sin: torch.Tensor, interleaved: bool = False):
        if cos_sin.dim() != 2 or cos_sin.dtype != torch.float32 or not cos_sin.is_contiguous():
            raise abi.AquaError(abi.AQUA_ERR_ARG, "cos_sin must be a contiguous f32 tensor [n_pos, rot_dim]")
        self.cos_sin = cos_sin
        self.desc = abi.aqua_rope(cos_sin.data_ptr(), cos_sin.shape[0], cos_sin.shape[1], int(bool(interleaved)))

    @classmethod
    def from_theta(cls, n_pos: int, theta: float = 500000.0, rot_dim: int = 128, interleaved: bool = False,
                   device="cuda") -> "AquaRope":
        """The usual table: angle i of position t is t * theta^(-2 i / rot_dim), formed in 64 bits."""
        inv = theta ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
        a = torch.arange(n_pos, dtype=torch.float64, device=device)[:, None] * inv
        return cls(torch.cat([a.cos(), a.sin()], 1).float().contiguous(), interleaved)
