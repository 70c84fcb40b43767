"""One-token attention over a paged cache in fp64 numpy, from the definition,
key by key through the block table: the oracle of fa_paged_decode."""
import numpy as np


def rows(pages, table_row, length, head):
    """The first `length` rows of one head, [n, d] fp64, and their key indexes:
    keys whose table entry names no page are left out."""
    num_pages, _, page_size, _ = pages.shape
    keys = [j for j in range(length)
            if j // page_size < len(table_row) and 0 <= table_row[j // page_size] < num_pages]
    at = np.array(keys, dtype=np.int64)
    if not len(at):
        return np.zeros((0, pages.shape[-1])), at
    page = np.asarray(table_row, dtype=np.int64)[at // page_size]
    return pages[page, head, at % page_size], at


def decode(q, k_pages, v_pages, table, kv_len, scale):
    """q [B, H, d], pages [P, H_kv, page, d] fp64 (already descaled). Returns
    o [B, H, d], lse [B, H], and what a bound on rounding errors needs: dev
    [B, H, d] = sum_j w_j |v_j - o| (w the softmax weights), flat [B, H, d] =
    sum_j |v_j - o| / sum_j exp(s_j - max s), mag [B, H] = max_j sum |q_i k_ji|,
    and absv [B, H, d] = sum_j w_j |v_j|."""
    B, H, d = q.shape
    group = H // k_pages.shape[1]
    o, dev, flat, absv = (np.zeros((B, H, d)) for _ in range(4))
    lse, mag = np.full((B, H), -np.inf), np.zeros((B, H))
    for b in range(B):
        for h in range(H):
            k, _ = rows(k_pages, table[b], int(kv_len[b]), h // group)
            v, _ = rows(v_pages, table[b], int(kv_len[b]), h // group)
            if not len(k):
                continue
            s = scale * (k @ q[b, h])
            e = np.exp(s - s.max())
            w = e / e.sum()
            lse[b, h] = s.max() + np.log(e.sum())
            o[b, h] = w @ v
            dev[b, h] = w @ np.abs(v - o[b, h])
            flat[b, h] = np.abs(v - o[b, h]).sum(0) / e.sum()
            absv[b, h] = w @ np.abs(v)
            mag[b, h] = (np.abs(k) @ np.abs(q[b, h])).max()
    return o, lse, dict(dev=dev, flat=flat, mag=mag, absv=absv)
