"""What a result of the attention over the 4-bit cache may differ by, checked on output and log.

Each element lies within the error of the kernels' arithmetic (``oracle.heads.attention_error``) and half an ulp of the
output's type; and the whole of a (sequence, head) within a share of its norm, since elements' errors do not add up:
2^-7 for bf16 (its rounding alone is at most 2^-8), 2^-16 for fp32."""
import numpy as np

from oracle import heads

HALF_ULP = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -23}
NORM = {"bf16": 2.0 ** -7, "fp32": 2.0 ** -16}


class Rejected(AssertionError):
    pass


def check(got, logs, q, rec, d, group, hq, scale, dtype, causal=True, window=0, many=False):
    """One sequence: results [n, hq, d] (and logs [n, hq] or None) for queries [n, hq, d] over records [kv, hk, words]."""
    k, v, ks, vs = heads.unpack(rec, d, group)
    g = hq // rec.shape[1]
    for h in range(hq):
        kh = h // g
        e, lse, _, _ = heads.attention(q[:, h], k[:, kh], v[:, kh], scale, causal, window)
        tol, log_tol = heads.attention_error(q[:, h], k[:, kh], v[:, kh], scale, causal, window, ks[:, kh], vs[:, kh],
                                             dtype, many)
        err = np.abs(got[:, h] - e)
        if not (err <= tol + HALF_ULP[dtype] * np.abs(e)).all():
            raise Rejected(f"head {h}: element, {np.nanmax(err / (tol + HALF_ULP[dtype] * np.abs(e) + 1e-300))}")
        if not np.linalg.norm(err) <= NORM[dtype] * np.linalg.norm(e):
            raise Rejected(f"head {h}: norm, {np.linalg.norm(err) / np.linalg.norm(e)}")
        if logs is not None:
            f = np.isfinite(lse)
            if not ((logs[:, h] == lse) | f).all() or not (np.abs(logs[f, h] - lse[f]) <= log_tol[f]).all():
                raise Rejected(f"head {h}: log")
