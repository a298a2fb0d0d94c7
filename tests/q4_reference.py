"""4-bit matrices for the tests: random ones in their own and in packed form, the packed layout from its description, the formulas of
strata_moe_linear and strata_moe_q4_experts in 64 bits, and how far fp32 sums may be off.

u = 2^-24 is half a step of fp32; the tensor core may cut where it adds, a whole step of 2u."""
import numpy as np
import torch

import ops_reference as ref
import quantized_routed_expert_top10_gb300 as qre
from ops_reference import U


class Matrices:
    """`count` matrices [n_out][d_in]; their weights are about d_in ** -0.5 large."""

    def __init__(self, count, n_out, d_in, group, zeros=False, scale_type=qre.BF16, paired=False, seed=1):
        g = torch.Generator().manual_seed(seed)
        self.count, self.n_out, self.d_in, self.group = count, n_out, d_in, group
        self.q = qre.q4(n_out, d_in, group, zeros=zeros, scale_type=scale_type, paired=paired)
        n = d_in // group
        self.codes = torch.randint(0, 256, (count, n_out, d_in // 2), dtype=torch.uint8, generator=g)
        self.scales = ((torch.rand(count, n_out, n, generator=g) + 0.5) * (d_in ** -0.5 / 4.6)).to(ref.TORCH[scale_type])
        self.zeros = torch.randint(0, 16, (count, n_out, n), dtype=torch.uint8, generator=g) if zeros else None

    def set_codes(self, q):
        """q: [count][n_out][d_in] whole numbers 0 .. 15."""
        q = torch.as_tensor(q, dtype=torch.uint8)
        self.codes = q[..., 0::2] | q[..., 1::2] << 4
        return self

    def weights(self, i):
        """Matrix i in 64 bits."""
        b = self.codes[i].numpy()
        q = np.stack((b & 15, b >> 4), -1).reshape(self.n_out, self.d_in).astype(np.float64)
        z = np.full((self.n_out, self.d_in // self.group), 8.0) if self.zeros is None else self.zeros[i].numpy().astype(np.float64)
        return (q - np.repeat(z, self.group, 1)) * np.repeat(ref.to64(self.scales[i]), self.group, 1)

    def packed_host(self):
        out = torch.full((self.count, qre.strata_q4_bytes(self.q)), 0xA5, dtype=torch.uint8)
        qre.strata_pack_q4(self.q, self.codes.contiguous(), self.scales, self.zeros, out, self.count)
        return out

    def packed(self, device):
        out = torch.full((self.count, qre.strata_q4_bytes(self.q)), 0xA5, dtype=torch.uint8, device=device)
        zeros = None if self.zeros is None else self.zeros.to(device)
        qre.strata_pack_q4_device(self.q, self.codes.contiguous().to(device), self.scales.to(device), zeros, out, self.count)
        return out


def packed_from_description(m, i):
    """The packed bytes of matrix i, element by element from the header's description."""
    b = m.codes[i].numpy()
    q = np.stack((b & 15, b >> 4), -1).reshape(m.n_out, m.d_in)
    s = m.scales[i].view(torch.int16).numpy().view(np.uint16)
    z = None if m.zeros is None else m.zeros[i].numpy()
    paired, n = bool(m.q.paired), m.d_in // m.group
    out = bytearray()
    for slab in range(-(-m.n_out // 16)):
        def row(r):
            if paired:
                return 8 * slab + r % 8 + (m.n_out // 2 if r >= 8 else 0)
            return 16 * slab + r if 16 * slab + r < m.n_out else None
        for chunk in range(-(-m.d_in // 128)):
            nb = min(4, (m.d_in - 128 * chunk) // 32)
            words = np.zeros((2, 32, nb), np.uint32)
            for half in range(2):
                for lane in range(32):
                    r = row(lane // 4 + 8 * half)
                    if r is None:
                        continue
                    for k in range(nb):
                        first = 128 * chunk + 32 * k + 8 * (lane % 4)
                        for j in range(4):
                            words[half, lane, k] |= np.uint32(int(q[r, first + 2 * j]) << 4 * j)
                            words[half, lane, k] |= np.uint32(int(q[r, first + 2 * j + 1]) << 16 + 4 * j)
            out += words.tobytes()
            per = 128 // m.group
            sc = np.zeros((8, per, 2), np.uint16)
            zp = np.zeros((8, max(per, 2), 2), np.uint8)
            for g in range(8):
                for k in range(per):
                    for half in range(2):
                        r, at = row(g + 8 * half), chunk * per + k
                        if r is not None and at < n:
                            sc[g, k, half] = s[r, at]
                            if z is not None:
                                zp[g, k, half] = z[r, at] & 15
            out += sc.tobytes()
            if z is not None:
                out += zp.tobytes()
    return np.frombuffer(bytes(out), np.uint8)


def additions(d_in, group):
    """Additions that may follow one another in a product's sum: an MMA adds 16 products to its sum (counted as two), a group's MMAs
    follow one another, then its scaled sum is added to the groups' (every chunk of a warp), then up to 16 warps' sums of 3 terms."""
    return 2 * (group // 16) + d_in // group + 48


def held(x, bits):
    """How far x [T][n] may be off when each row's 128 columns are held with `bits` bits, down to 2^-40 of the largest (half a step)."""
    T, n = x.shape
    full = np.zeros((T, -(-n // 128) * 128))
    full[:, :n] = np.abs(x)
    top = np.repeat(full.reshape(T, -1, 128).max(2), 128, 1)[:, :n]
    return 2.0 ** -bits * np.abs(x) + 2.0 ** -39 * top


def product(x, x_err, w, adds):
    """x w^T [T][n] in 64 bits, and how far fp32 may be off it when x is off by x_err."""
    return x @ w.T, x_err @ np.abs(w).T + adds * 2 * U * ((np.abs(x) + x_err) @ np.abs(w).T)


def experts(x, gate_up, down, ids, weights, out_kind, x_kind=qre.F32):
    """out [T][d_model] in 64 bits and how far fp32 may be off; x [T][d_model]."""
    T, k = ids.shape
    d_ff, n = down.d_in, down.n_out
    out, err = np.zeros((T, n)), np.zeros((T, n))
    size = np.zeros((T, n))
    for e in np.unique(ids[ids >= 0]):
        t, i = np.nonzero((ids == e) & (weights != 0))
        if len(t) == 0:
            continue
        gu, gu_err = product(x[t], held(x[t], 22 if x_kind == qre.F32 else 60), gate_up.weights(int(e)), additions(gate_up.d_in, gate_up.group))
        g, u, g_err, u_err = gu[:, :d_ff], gu[:, d_ff:], gu_err[:, :d_ff], gu_err[:, d_ff:]
        with np.errstate(over="ignore"):
            silu = g / (1.0 + np.exp(-g))
        h = silu * u
        # |silu'| < 1.1; an exponential (4 u), a sum, a quotient, a product
        h_err = 1.1 * g_err * (np.abs(u) + u_err) + np.abs(silu) * u_err + 8 * U * np.abs(h)
        h_err = h_err + held(h, 11 if out_kind == qre.BF16 else 22)
        part, part_err = product(h, h_err, down.weights(int(e)), additions(down.d_in, down.group))
        w = weights[t, i][:, None]
        np.add.at(out, t, w * part)
        np.add.at(err, t, np.abs(w) * part_err)
        np.add.at(size, t, np.abs(w * part))
    return out, err + (k + 1) * U * (size + err)
