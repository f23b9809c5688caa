"""Oracle of the paged cache's tables, one token and one page at a time, on Python lists."""
from __future__ import annotations


def extend(table, lens, stack, count, new_rows, page_size, rows):
    """Lengthens sequences in place.  Returns (count, cu_rows, slots, positions, [why each was not served, or None])."""
    cu, slots, positions, why = [0], [], [], []
    num_pages, width = len(stack), len(table[0])
    need_all = rows_all = 0
    free, free_now = count, count
    for b, n in enumerate(new_rows):
        old = lens[b]
        if old < 0 or n < 0 or old + n > width * page_size:
            why.append("batch")
            cu.append(cu[-1])
            continue
        need = -(-(old + n) // page_size) - -(-old // page_size)
        need_all += need
        rows_all += n
        if rows_all > rows:
            why.append("batch" if n else None)
        elif need and need_all > free:
            why.append("pages")
        else:
            why.append(None)
            for pos in range(old, old + n):
                if pos % page_size == 0:
                    free_now -= 1
                    page = stack[free_now]
                    table[b][pos // page_size] = page if 0 <= page < num_pages else -1
                page = table[b][pos // page_size]
                slots.append(page * page_size + pos % page_size if 0 <= page < num_pages else -1)
                positions.append(pos)
            lens[b] = old + n
        cu.append(len(slots))
    return free_now, cu, slots, positions, why


def release(table, lens, stack, count, done, page_size):
    """Ends sequences in place.  Returns (count, whether all that was given back was a page that the stack could hold)."""
    num_pages, width = len(stack), len(table[0])
    fine = True
    for b, d in enumerate(done):
        if not d:
            continue
        fine = fine and 0 <= lens[b] <= width * page_size
        held = -(-min(max(lens[b], 0), width * page_size) // page_size)
        for k in range(held):
            page = table[b][k]
            if 0 <= page < num_pages and count < num_pages:
                stack[count] = page
                count += 1
            else:
                fine = False
            table[b][k] = -1
        lens[b] = 0
    return count, fine
