"""Calls about pages from several host threads (needs a GB300)."""
import threading

import pytest
import torch

from exact_attention_57_gb300 import fa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("op", ["free", "compact"])
def test_threads_with_caches_of_different_sizes(op):
    """Two threads sweep caches of 8M and 4M blocks over and over, each on a stream of
    its own: no call is refused and every result is right."""
    sizes, failed = (1 << 23, 1 << 22), []

    def work(blocks):
        try:
            stream = torch.cuda.Stream()
            s = stream.cuda_stream
            with torch.cuda.stream(stream):
                table = torch.tensor([[blocks - 1, 0, 77]], dtype=torch.int32, device=DEV)
                lens = torch.tensor([33], dtype=torch.int32, device=DEV)
                ids = torch.empty(blocks, dtype=torch.int32, device=DEV)
                out, counts = (torch.empty(3, dtype=torch.int32, device=DEV) for _ in range(2))
                n = fa.fa_kv_compact_workspace(blocks)
                ws = torch.empty(n, dtype=torch.uint8, device=DEV)
                for i in range(600):
                    if op == "free":
                        st = fa.fa_kv_free(table.data_ptr(), lens.data_ptr(), None, ids.data_ptr(),
                                           out.data_ptr(), 1, 3, 16, blocks, s)
                    else:
                        st = fa.fa_kv_compact(table.data_ptr(), lens.data_ptr(), out.data_ptr(),
                                              ids.data_ptr(), counts.data_ptr(), 1, 3, 16, blocks,
                                              [], [], ws.data_ptr(), n, s)
                    if st != fa.FA_OK:
                        failed.append((blocks, i, fa.fa_status_string(st)))
                        return
                stream.synchronize()
                if op == "free":
                    ok = out[0].item() == 3 and ids[:3].tolist() == [-1] * 3
                    want = torch.arange(blocks, dtype=torch.int32, device=DEV)
                    keep = torch.ones(blocks, dtype=torch.bool, device=DEV)
                    keep[[0, 77, blocks - 1]] = False
                    ok = ok and torch.equal(ids[3:], want[keep])
                else:
                    # blocks 0, 77 and the last: 77 and the last move to 1 and 2
                    ok = out.tolist() == [2, 0, 1] and ids[0] == 0 and ids[77] == 1 and ids[-1] == 2
                    ok = ok and int((ids >= 0).sum()) == 3
                if not ok:
                    failed.append((blocks, "wrong"))
        except Exception as e:
            failed.append((blocks, repr(e)))

    threads = [threading.Thread(target=work, args=(n,)) for n in sizes]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
