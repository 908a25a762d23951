"""Rules of the latent attention's sources that no run can show without a
failing GPU: they are read from the text."""
import os
import re

import sparse_attention_top_idx_gb300 as pkg

CSRC = os.path.join(os.path.dirname(pkg.__file__), "csrc")


def source(name):
    """A source file without its comments."""
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


def softmax_role():
    """The absorbed kernel's softmax role: its loop over the pieces."""
    text = source("latent_attend.cu")
    role = text[text.index("else if (warp >= 4)"):text.index("if (kCl > 1 && it == 0")]
    return role[role.index("while (ok && walk.next(p, w))"):]


def test_softmax_threads_leave_together():
    """The role's named barriers count every softmax thread.  A bounded wait may
    run out in some of them alone, so a thread may leave the loops only where
    all of them vote (named_any), or where none is missing: at the end of a
    cluster's only piece."""
    role = softmax_role()
    votes = re.findall(r"if \(named_any<1, kSoftThreads>\(!ok\)\) \{ ok = false; break; \}", role)
    assert len(votes) == 2
    rest = role.replace(votes[0], "")
    left = [m.group(1).strip() for m in re.finditer(r"([^;{}]*)\bbreak;", rest)]
    assert left == [""], left                   # the cluster's, unconditional
    assert not re.search(r"if \(!ok\)|\breturn\b|\bgoto\b", rest)
